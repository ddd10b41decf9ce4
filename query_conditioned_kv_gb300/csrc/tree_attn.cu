// tree_attn.cu — attention of drafted token trees over a paged KV cache, one
// layer.  Row i of request r sees the c cached positions and the nodes its
// mask marks:
//   z_p = scale·q·k_p,  lse = ln Σ_p exp z_p,  out = Σ_p exp(z_p − lse)·v_p
#include <math.h>

#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
  const uint16_t *q, *kpool, *vpool;
  const int32_t *block_table, *ctx_len, *q_off;
  const uint32_t *mask;  // [n_q][mask_words] or NULL (a chain)
  uint16_t *out;
  float *lse;
  int32_t *status;
  int64_t n_slots;
  int max_blocks, mask_words, n_req, n_q, max_tree, H, Hq, G, BS;
  float zscale;  // scale·log2(e)
};

// Request r's sizes; false (recorded by the caller that passes record) when
// they are out of range.
__device__ __forceinline__ bool tree_request(const TreeArgs &a, int r, bool record, int &c, int &q0,
                                             int &T) {
  c = a.ctx_len[r];
  q0 = a.q_off[r];
  const int64_t t = (int64_t)a.q_off[r + 1] - q0;
  T = (int)t;
  const bool ok = c >= 0 && q0 >= 0 && t >= 0 && t <= a.max_tree && q0 + t <= a.n_q &&
                  c + t <= (int64_t)a.max_blocks * a.BS;
  if (!ok && record) record_error(a.status, KVC_ERR_BOUNDS);
  return ok;
}

// One warp per (node, query head); lanes split D, an online softmax over the
// positions in order.
template <int D>
__global__ void __launch_bounds__(128)
k_tree_attn(TreeArgs a) {
  constexpr int E = D / 32;
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  const int hq = blockIdx.z * 4 + (threadIdx.x >> 5), i = blockIdx.x;
  int c, q0, T;
  const bool ok = tree_request(a, r, i == 0 && hq == 0 && lane == 0, c, q0, T);
  if (!ok || i >= T || hq >= a.Hq) return;
  const int h = hq / a.G;
  const int64_t row = (int64_t)(q0 + i) * a.Hq + hq;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; e++) {
    q[e] = bf16_lo(a.q[row * D + lane * E + e]);
    o[e] = 0.f;
  }
  const int64_t n_blocks = a.n_slots / a.BS;
  for (int p = 0; p < c + T; p++) {
    if (p >= c) {
      const int j = p - c;
      const bool see = a.mask ? (a.mask[(int64_t)(q0 + i) * a.mask_words + j / 32] >> (j % 32)) & 1
                              : j <= i;
      if (!see) continue;
    }
    const int32_t b = a.block_table[(int64_t)r * a.max_blocks + p / a.BS];
    if (b < 0 || b >= n_blocks) {
      if (lane == 0) record_error(a.status, KVC_ERR_BOUNDS);
      continue;
    }
    const int64_t at = (((int64_t)b * a.BS + p % a.BS) * a.H + h) * D + lane * E;
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) z = fmaf(q[e], bf16_lo(a.kpool[at + e]), z);
#pragma unroll
    for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
    z *= a.zscale;
    const float m2 = fmaxf(m, z), f = exp2f(m - m2), w = exp2f(z - m2);
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; e++) o[e] = o[e] * f + w * bf16_lo(a.vpool[at + e]);
    m = m2;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; e++) {
    const __nv_bfloat16 v = __float2bfloat16(m == -INFINITY ? 0.f : o[e] * inv);
    a.out[row * D + lane * E + e] = *reinterpret_cast<const uint16_t *>(&v);
  }
  if (lane == 0) a.lse[row] = m == -INFINITY ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

size_t tree_attn_ws_bytes(int, int, int, int, int, int, int) { return 16; }

cudaError_t launch_tree_attn(const uint16_t *q, const uint16_t *kpool, const uint16_t *vpool,
                             int64_t n_slots, const int32_t *block_table, int max_blocks,
                             const int32_t *ctx_len, const int32_t *q_off,
                             const uint32_t *tree_mask, int mask_words, int n_req, int n_q,
                             int max_tree, int H, int Hq, int D, int BS, float scale,
                             uint16_t *out, float *lse, void *, int32_t *status,
                             cudaStream_t s) {
  TreeArgs a{q,   kpool,   vpool,      block_table, ctx_len, q_off, tree_mask, out,
             lse, status,  n_slots,    max_blocks,  mask_words, n_req, n_q,    max_tree,
             H,   Hq,      Hq / H,     BS,          scale * kLog2e};
  const dim3 grid(max_tree, n_req, (Hq + 3) / 4);
  if (D == 128) k_tree_attn<128><<<grid, 128, 0, s>>>(a);
  else k_tree_attn<64><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
