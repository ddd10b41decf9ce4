// prompt_attn.cu — causal attention of the new rows of packed prompts over a
// paged cache that already holds their keys and values, one layer.  Row i of
// request r sees the positions 0 … c + i:
//   z_p = scale·q·k_p,  lse = ln Σ_p exp z_p,  out = Σ_p exp(z_p − lse)·v_p
//
// The rows of a KV head are (token, head of the group) pairs, token by token: a
// tile of them shares its keys whatever the group's size, and is causal in steps
// of G rows.
//
// k_prompt_rows: a CTA takes 64 rows of one KV head, a warp 16 of them; tiles of 64
// keys pass through two cp.async buffers, and mma.sync m16n8k16 makes both products.
#include <algorithm>

#include "tree_rows.cuh"

namespace kvc {
namespace {

constexpr int kPrWarps = 4;
constexpr int kPrThreads = kPrWarps * 32;
constexpr int kPrKeys = 64;

template <int D>
__global__ void __launch_bounds__(kPrThreads, 2)
k_prompt_rows(TreeArgs a) {
  constexpr int KS = D / 16, NT = D / 8, CH = D / 8, HK = kPrKeys / 32;
  constexpr uint32_t kTile = kPrKeys * D * 2;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ uint32_t ok_s[2][HK];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(sm);
  const int r = blockIdx.z, h = blockIdx.y;
  int c, q0, T;
  if (!tree_request(a, r, c, q0, T)) {
    if (blockIdx.x == 0 && h == 0 && tid == 0) record_error(a.status, KVC_ERR_BOUNDS);
    return;
  }
  // (the last rows first: they see the most)
  const int rt = (int)gridDim.x - 1 - blockIdx.x;
  if ((int64_t)rt * 64 >= (int64_t)T * a.G) return;
  const int n_rows = min(64, T * a.G - rt * 64), wrt = rt * 4 + warp;
  const int end = c + (rt * 64 + n_rows - 1) / a.G + 1;  // positions some row sees
  const int n_kt = (end + kPrKeys - 1) / kPrKeys;
  const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
  const int64_t n_blocks = a.n_slots / a.BS;

  auto issue = [&](int t, int st) {
    constexpr int RPW = kPrKeys / kPrWarps, RPI = 32 / CH;  // rows of a warp, of an instruction
    int32_t slot = -1;
    const int p = t * kPrKeys + warp * RPW + (lane % RPW);
    if (p < end) {
      const int pg = page_of(p, a.bs_inv);
      const int32_t b = bt[pg];
      if (b >= 0 && b < n_blocks) slot = b * a.BS + p - pg * a.BS;
      else record_error(a.status, KVC_ERR_BOUNDS);
    }
    const uint32_t ok = __ballot_sync(0xFFFFFFFFu, slot >= 0) & 0xFFFFu;
    if (lane == 0) reinterpret_cast<uint16_t *>(ok_s[st])[warp] = (uint16_t)ok;
    const uint32_t dst = base + st * 2 * kTile;
    const int col = lane % CH;
#pragma unroll
    for (int i = 0; i < RPW / RPI; i++) {
      const int row = i * RPI + lane / CH;
      const int32_t sl = __shfl_sync(0xFFFFFFFFu, slot, row);
      const int64_t from = ((int64_t)max(sl, 0) * a.H + h) * D + col * 8;
      cp_async16(dst + swz<D>(warp * RPW + row, col), a.kpool + from, sl >= 0);
      cp_async16(dst + kTile + swz<D>(warp * RPW + row, col), a.vpool + from, sl >= 0);
    }
  };
  issue(0, 0);
  cp_commit();
  uint32_t qf[KS][4];
#pragma unroll
  for (int hf = 0; hf < 2; hf++) {
    const int row = warp * 16 + hf * 8 + lane / 4, x = rt * 64 + row;
    const uint16_t *p =
        a.q + ((int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G) * D + 2 * (lane % 4);
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
      qf[ks][hf] = row < n_rows ? __ldg(reinterpret_cast<const uint32_t *>(p + 16 * ks)) : 0u;
      qf[ks][2 + hf] = row < n_rows ? __ldg(reinterpret_cast<const uint32_t *>(p + 16 * ks + 8)) : 0u;
    }
  }
  float o[1][NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < NT; n++) o[0][n][0] = o[0][n][1] = o[0][n][2] = o[0][n][3] = 0.f;

  for (int t = 0; t < n_kt; t++) {
    if (t + 1 < n_kt) issue(t + 1, (t + 1) & 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    const uint32_t kb = base + (t & 1) * 2 * kTile, vb = kb + kTile;
#pragma unroll
    for (int half = 0; half < HK; half++) {
      const int p0 = t * kPrKeys + half * 32;
      const uint32_t okb = ok_s[t & 1][half];
      const uint32_t kh = kb + half * 32 * D * 2;
      float s[1][4][4];
#pragma unroll
      for (int n = 0; n < 4; n++) s[0][n][0] = s[0][n][1] = s[0][n][2] = s[0][n][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
          uint32_t b[4];
          ldsm4(kh + swz<D>(kk * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), b);
          mma16816(s[0][2 * kk], qf[ks], b[0], b[1]);
          mma16816(s[0][2 * kk + 1], qf[ks], b[2], b[3]);
        }
      const bool masked = p0 + 32 > c || okb != 0xFFFFFFFFu;
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        uint32_t vis = 0xFFFFFFFFu;
        if (masked) {
          const int x = wrt * 16 + hf * 8 + lane / 4;
          vis = x < T * a.G ? visible_bits<32>(a, x / a.G, q0, c, T, p0) & okb : 0u;
        }
        float mx = m[hf];
#pragma unroll
        for (int n = 0; n < 4; n++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float z = s[0][n][hf * 2 + e] * a.zscale;
            if (!((vis >> (n * 8 + 2 * (lane % 4) + e)) & 1u)) z = -INFINITY;
            s[0][n][hf * 2 + e] = z;
            mx = fmaxf(mx, z);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const float ref = mx == -INFINITY ? 0.f : mx, f = ex2(m[hf] - ref);
        m[hf] = mx;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 4; n++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const float w = ex2(s[0][n][hf * 2 + e] - ref);
            s[0][n][hf * 2 + e] = w;
            sum += w;
          }
        l[hf] = l[hf] * f + sum;
#pragma unroll
        for (int n = 0; n < NT; n++) {
          o[0][n][hf * 2] *= f;
          o[0][n][hf * 2 + 1] *= f;
        }
      }
      tile_values<D, 1, 32>(a, s, o, vb + half * 32 * D * 2, okb, wrt, q0, c, T, p0);
    }
    __syncthreads();
  }
#pragma unroll
  for (int hf = 0; hf < 2; hf++) {
    float sum = l[hf];
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    const int row = warp * 16 + hf * 8 + lane / 4, x = rt * 64 + row;
    if (row >= n_rows) continue;
    const int64_t qr = (int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int n = 0; n < NT; n++)
      *reinterpret_cast<uint32_t *>(a.out + qr * D + n * 8 + 2 * (lane % 4)) =
          pack_bf16x2(o[0][n][hf * 2] * inv, o[0][n][hf * 2 + 1] * inv);
    if (lane % 4 == 0) a.lse[qr] = sum == 0.f ? -INFINITY : (m[hf] + log2f(sum)) * kLn2;
  }
}

}  // namespace

cudaError_t launch_prompt_attn(const uint16_t *q, const uint16_t *kpool, const uint16_t *vpool,
                               int64_t n_slots, const int32_t *block_table, int max_blocks,
                               const int32_t *ctx_len, const int32_t *q_off, int n_req, int n_q,
                               int max_rows, int H, int Hq, int D, int BS, float scale,
                               uint16_t *out, float *lse, int32_t *status, cudaStream_t s) {
  TreeArgs a{};
  a.q = q, a.kpool = kpool, a.vpool = vpool, a.block_table = block_table;
  a.ctx_len = ctx_len, a.q_off = q_off, a.out = out, a.lse = lse, a.status = status;
  a.n_slots = n_slots, a.max_blocks = max_blocks, a.n_req = n_req, a.n_q = n_q;
  a.max_tree = max_rows, a.H = H, a.Hq = Hq, a.G = Hq / H, a.BS = BS, a.bs_inv = page_inverse(BS);
  a.rstep = 16;
  a.zscale = scale != 0.f ? scale * kLog2e : 1e-30f;  // (so that −inf stays −inf when scaled)
  auto *kern = D == 128 ? k_prompt_rows<128> : k_prompt_rows<64>;
  const int smem = 4 * kPrKeys * D * 2;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(((int64_t)max_rows * a.G + 63) / 64), (unsigned)H, (unsigned)n_req);
  kern<<<grid, kPrThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
