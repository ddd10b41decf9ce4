// tree_commit.cu — commit of the accepted path of a drafted token tree: the
// accepted nodes' K and V rows move, in place, to the positions that follow
// the cache, every layer and KV head.
//
// For request r with c cached positions and accepted nodes a_0 < a_1 < …,
// position c + a_i → c + i.  Since a is ascending, a_i ≥ i and every later
// source a_j (j > i) is above i: a thread that owns one 16-byte column and
// walks i upwards never overwrites a row it still has to read, also when it
// reads four rows ahead of the first write.  So one pass over the rows, no
// scratch, and the columns are independent.
//
// What bounds it: latency.  A path of 8 rows of 2 KB (8 KV heads, D 128) is
// 64 KB of traffic a layer; a thread reads four rows before it writes the first
// (eight take the registers of two more CTAs per SM: 12.0 us against 10.4 for 64
// paths whose rows are in L2, the same otherwise).  Measured: 36 layers, 8 KV
// heads, D 128: one path of 5 nodes 8 us with the call, 64 paths of up to 8
// nodes 17 us, 3.9 TB/s.
#include <algorithm>

#include "kvc_internal.cuh"
#include "mma_ptx.cuh"

namespace kvc {
namespace {

constexpr int kCommitThreads = 256;
constexpr int kCommitAhead = 4;  // rows read before the first of them is written

struct CommitArgs {
  uint16_t *kpool, *vpool;      // [L][n_slots][H][D]
  const int32_t *block_table;   // [n_req][max_blocks]
  const int32_t *ctx_len, *q_off, *path, *n_path;
  int32_t *seq_out, *row_idx, *row_vis, *status;
  int64_t n_slots;
  int max_blocks, max_path, row_elems, BS;  // row_elems = H·D
  int L, layers;                            // layers of one CTA
  uint32_t bs_inv;                          // page_inverse(BS)
};

__global__ void __launch_bounds__(kCommitThreads, 6)
k_tree_commit(CommitArgs a) {
  extern __shared__ int32_t s_slot[];  // [2][max_path]: source, destination (−1: no copy)
  const int r = blockIdx.x, tid = threadIdx.x;
  const int c = a.ctx_len[r], q0 = a.q_off[r], n = a.n_path[r];
  const int64_t T = (int64_t)a.q_off[r + 1] - q0;
  const int64_t cap = (int64_t)a.max_blocks * a.BS;
  const int32_t *path = a.path + (int64_t)r * a.max_path;
  // (asked for with the sizes, so that the loops below find it in L1)
  if (tid < a.max_path) asm volatile("prefetch.global.L1 [%0];" ::"l"(path + tid));
  bool bad = c < 0 || q0 < 0 || T < 0 || c + T > cap || n < 0 || n > a.max_path || n > T;
  if (!bad)
    for (int i = tid; i < n; i += kCommitThreads) {
      const int p = path[i];
      if (p < 0 || p >= T || (i > 0 && p <= path[i - 1])) bad = true;
    }
  bad = __syncthreads_or(bad);
  if (blockIdx.y == 0) {
    if (tid == 0) {
      a.seq_out[r] = bad ? max(c, 0) : c + n;
      if (bad) record_error(a.status, KVC_ERR_BOUNDS);
    }
    for (int i = tid; i < a.max_path; i += kCommitThreads) {
      const bool on = !bad && i < n;
      if (a.row_idx) a.row_idx[(int64_t)r * a.max_path + i] = on ? q0 + path[i] : 0;
      if (a.row_vis) a.row_vis[(int64_t)r * a.max_path + i] = on ? c + i + 1 : 0;
    }
  }
  if (bad) return;
  const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
  const int64_t n_blocks = a.n_slots / a.BS;
  int32_t *src = s_slot, *dst = s_slot + a.max_path;
  for (int i = tid; i < n; i += kCommitThreads) {
    const int p = c + path[i], d = c + i;
    const int gp = page_of(p, a.bs_inv), gd = page_of(d, a.bs_inv);
    const int32_t bp = bt[gp], bd = bt[gd];
    const bool ok = bp >= 0 && bp < n_blocks && bd >= 0 && bd < n_blocks;
    if (!ok) record_error(a.status, KVC_ERR_BOUNDS);
    src[i] = bp * a.BS + p - gp * a.BS;
    dst[i] = ok && p != d ? bd * a.BS + d - gd * a.BS : -1;
  }
  __syncthreads();
  const int l0 = blockIdx.y * a.layers, n_l = min(a.layers, a.L - l0);
  const int cols = a.row_elems / 8;  // 16-byte columns of one row
  for (int x = tid; x < 2 * cols * n_l; x += kCommitThreads) {
    const int l = x / (2 * cols), t = x - l * 2 * cols;
    const int64_t layer = (int64_t)(l0 + l) * a.n_slots;
    uint16_t *pool = t < cols ? a.kpool : a.vpool;
    const int col = (t < cols ? t : t - cols) * 8;
    for (int i0 = 0; i0 < n; i0 += kCommitAhead) {
      uint4 v[kCommitAhead];
#pragma unroll
      for (int k = 0; k < kCommitAhead; k++)
        if (i0 + k < n && dst[i0 + k] >= 0)
          v[k] = *reinterpret_cast<const uint4 *>(pool + (layer + src[i0 + k]) * a.row_elems + col);
#pragma unroll
      for (int k = 0; k < kCommitAhead; k++)
        if (i0 + k < n && dst[i0 + k] >= 0)
          *reinterpret_cast<uint4 *>(pool + (layer + dst[i0 + k]) * a.row_elems + col) = v[k];
    }
  }
}

}  // namespace

cudaError_t launch_tree_commit(uint16_t *kpool, uint16_t *vpool, int64_t n_slots,
                               const int32_t *block_table, int max_blocks,
                               const int32_t *ctx_len, const int32_t *q_off,
                               const int32_t *path, const int32_t *n_path, int max_path,
                               int n_req, int L, int H, int D, int BS, int32_t *seq_out,
                               int32_t *row_idx, int32_t *row_vis, int32_t *status,
                               cudaStream_t s) {
  CommitArgs a{kpool,   vpool,   block_table, ctx_len, q_off, path,       n_path,
               seq_out, row_idx, row_vis,     status,  n_slots, max_blocks, max_path,
               H * D,   BS};
  // one CTA a layer until the GPU is full (6 CTAs of 256 threads an SM), then several
  // layers a CTA, which share the lookups
  const int64_t full = 6 * (int64_t)device_sm_count();
  a.L = L;
  a.layers = (int)std::min<int64_t>(L, ((int64_t)n_req * L + full - 1) / full);
  a.bs_inv = page_inverse(BS);
  k_tree_commit<<<dim3(n_req, (L + a.layers - 1) / a.layers), kCommitThreads, 2 * max_path * sizeof(int32_t), s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
