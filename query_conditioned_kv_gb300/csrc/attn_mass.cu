// attn_mass.cu — accumulated attention weight per (layer, request, KV head,
// cached position): the rows' softmax weights, recovered from attention's
// LSE, added up over the rows and the heads of the group,
//   mass[p] ← (p < n_mass ? decay·mass[p] : 0)
//             + Σ_{rows i, p < vis_i} Σ_g exp(scale·q_{i,g}·k_p − lse_{i,g})
#include <math.h>

#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct MassArgs {
  const uint16_t *q, *kpool;  // [L][n_q][Hq][D], [L][n_slots][H][D]
  const float *lse;           // [L][n_q][Hq]
  const int32_t *row_idx, *row_vis, *row_off, *block_table, *seqused, *n_mass;
  float *mass;
  int32_t *status;
  int64_t n_slots;
  int n_q, n_rows, max_rows, max_blocks, cap, n_req, L, H, Hq, G, BS;
  float zscale, decay;
};

// One warp per position; lanes split D.
template <int D>
__global__ void __launch_bounds__(256)
k_attn_mass(MassArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int p = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int seg = blockIdx.y + gridDim.y * blockIdx.z;
  if (seg >= a.L * a.n_req * a.H) return;
  const int h = seg % a.H, r = (seg / a.H) % a.n_req;
  const int64_t l = seg / (a.H * a.n_req);
  const int seq = a.seqused[r], r0 = a.row_off[r], r1 = a.row_off[r + 1];
  if (seq < 0 || seq > a.cap || r0 < 0 || r1 < r0 || r1 > a.n_rows || r1 - r0 > a.max_rows) {
    if (lane == 0) record_error(a.status, KVC_ERR_BOUNDS);
    return;
  }
  if (p >= seq) return;
  const int32_t b = a.block_table[(int64_t)r * a.max_blocks + p / a.BS];
  float sum = 0.f;
  if (b < 0 || b >= a.n_slots / a.BS) {
    if (lane == 0) record_error(a.status, KVC_ERR_BOUNDS);
  } else {
    const int64_t at =
        ((l * a.n_slots + (int64_t)b * a.BS + p % a.BS) * a.H + h) * D + lane * E;
    float k[E];
#pragma unroll
    for (int e = 0; e < E; e++) k[e] = bf16_lo(a.kpool[at + e]);
    for (int i = r0; i < r1; i++) {
      if (p >= a.row_vis[i]) continue;
      const int x = a.row_idx ? a.row_idx[i] : i;
      if (x < 0 || x >= a.n_q) {
        if (lane == 0) record_error(a.status, KVC_ERR_BOUNDS);
        continue;
      }
      for (int g = 0; g < a.G; g++) {
        const int64_t row = (l * a.n_q + x) * a.Hq + h * a.G + g;
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < E; e++) z = fmaf(bf16_lo(a.q[row * D + lane * E + e]), k[e], z);
#pragma unroll
        for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
        const float lse = a.lse[row];
        if (lse != -INFINITY) sum += exp2f(fmaf(z, a.zscale, -lse * kLog2e));
      }
    }
  }
  if (lane == 0) {
    float *m = a.mass + (int64_t)seg * a.cap + p;
    *m = (p < a.n_mass[r] ? a.decay * *m : 0.f) + sum;
  }
}

}  // namespace

size_t attn_mass_ws_bytes(int, int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_attn_mass(const uint16_t *q, const float *lse, int n_q,
                             const int32_t *row_idx, const int32_t *row_vis,
                             const int32_t *row_off, int n_rows, int max_rows,
                             const uint16_t *kpool, int64_t n_slots,
                             const int32_t *block_table, int max_blocks,
                             const int32_t *seqused, const int32_t *n_mass, int n_req, int L,
                             int H, int Hq, int D, int BS, float scale, float decay, float *mass,
                             void *, int32_t *status, cudaStream_t s) {
  MassArgs a{q,      kpool,   lse,    row_idx,  row_vis,    row_off,         block_table, seqused,
             n_mass, mass,    status, n_slots,  n_q,        n_rows,          max_rows,    max_blocks,
             max_blocks * BS, n_req,  L,        H,          Hq,              Hq / H,      BS,
             scale * kLog2e,  decay};
  const int segs = L * n_req * H, y = segs < 32768 ? segs : 32768;
  const dim3 grid((a.cap + 7) / 8, y, (segs + y - 1) / y);
  if (D == 128) k_attn_mass<128><<<grid, 256, 0, s>>>(a);
  else k_attn_mass<64><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
