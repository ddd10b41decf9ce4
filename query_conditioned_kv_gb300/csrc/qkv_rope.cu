// qkv_rope.cu — a layer's new tokens on their way into the paged cache: per
// head, queries and keys are normed (y = x·w / sqrt(mean x² + eps)), rotated by
// their position's table row and rounded once; keys and values go to their
// slots.
//
// Bound by HBM: every row is read once and written once, and nothing else is
// of that size (a token's table row serves all its heads and is read once).
// A warp owns a token (or a part of its heads, where there are few tokens):
// D/16 lanes hold a head, lane c the pairs (j, j + D/2) for j in [8c, 8c + 8),
// so that a rotation needs no exchange and the norm only D/16 lanes'.  Its
// cosines and sines stay in registers over all heads.  What counts is how many
// warps an SM holds (a warp waits for lookups, its row and the norm's sum in turn) and
// how many instructions a row takes, so columns go in pairs through packed products:
// 28 warps with one group of heads ahead take 41 us for 8192 tokens of 48 heads with
// norms and raw keys (222 MB, 5.40 TB/s) and 125 us for 22K tokens of 64 heads without
// (6.10 TB/s, 90 % of a copy's rate).  24 warps take 45 and 129, 30 to 32 warps 43 and
// 125; one column an instruction, 32 warps, 43 and 127; that with 24 warps and two
// groups ahead 52 and 143, with bulk copies into a ring of shared memory 47 and 137.
#include "kvc_internal.cuh"
#include "tc_ptx.cuh"

namespace kvc {
namespace {

using namespace tc;

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack2(uint64_t x) {
  float a, b;
  upk2(x, a, b);
  return pack_bf16x2(a, b);
}

constexpr int kRopeWarps = 2;
constexpr int kRopeCtas = 14;  // per SM
constexpr int kAhead = 1;    // groups of heads in flight

struct RopeArgs {
  const uint16_t *q, *k, *v, *wq, *wk;
  const float *tab;
  const int32_t *pos, *q_off, *ctx_len, *block_table;
  uint16_t *q_out, *kpool, *vpool, *k_raw;
  int32_t *status;
  int64_t qs, ks, vs, raw_stride, n_slots;
  float eps;
  int n_tok, n_pos, n_req, max_blocks, H, Hq, BS;
};

// Request r's sizes; false when they are out of range.
__device__ __forceinline__ bool rope_request(const RopeArgs &a, int r, int &c, int &q0, int &T) {
  c = a.ctx_len[r];
  q0 = a.q_off[r];
  const int64_t t = (int64_t)a.q_off[r + 1] - q0;
  T = (int)t;
  return c >= 0 && q0 >= 0 && t >= 0 && q0 + t <= a.n_tok &&
         c + t <= (int64_t)a.max_blocks * a.BS;
}

// The last r with off[r] ≤ x (off ascending, n + 1 entries), −1 if none; by a
// whole warp, a 32nd of the range a step.
__device__ __forceinline__ int warp_last_le(const int32_t *off, int n, int x) {
  const int lane = threadIdx.x & 31;
  int base = 0, len = n + 1;
  for (;;) {
    const int step = (len + 31) / 32;
    const int64_t i = (int64_t)lane * step;
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, i < len && off[base + i] <= x);
    if (!b) return -1;
    const int at = (31 - __clz(b)) * step;
    base += at;
    if (step == 1) return base;
    len = min(step, len - at);
  }
}

template <int D>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeCtas)
k_qkv_rope(RopeArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH, HALF = D / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0)  // one report per bad request
    for (int r = threadIdx.x; r < a.n_req; r += kRopeWarps * 32) {
      int c, q0, T;
      if (!rope_request(a, r, c, q0, T)) record_error(a.status, KVC_ERR_BOUNDS);
    }
  const int x = blockIdx.x * kRopeWarps + warp;
  if (x >= a.n_tok) return;
  // (parts of a token's heads: groups of HPW, an even share each)
  const int heads = a.Hq + 2 * a.H, groups = (heads + HPW - 1) / HPW;
  const int g0 = groups * (int)blockIdx.y / (int)gridDim.y;
  const int g1 = groups * ((int)blockIdx.y + 1) / (int)gridDim.y;
  const int sub = lane / LPH, c = lane % LPH;

  auto source = [&](int hh) -> const uint16_t * {
    return hh < a.Hq          ? a.q + x * a.qs + (int64_t)hh * D
           : hh < a.Hq + a.H ? a.k + x * a.ks + (int64_t)(hh - a.Hq) * D
                             : a.v + x * a.vs + (int64_t)(hh - a.Hq - a.H) * D;
  };
  uint4 lo[kAhead], hi[kAhead];
  auto load = [&](int u, int g) {
    const int hh = g * HPW + sub;
    if (g < g1 && hh < heads) {
      const uint16_t *p = source(hh);
      lo[u] = ld_stream(p + 8 * c);
      hi[u] = ld_stream(p + HALF + 8 * c);
    }
  };
#pragma unroll
  for (int u = 0; u < kAhead; u++) load(u, g0 + u);

  // where the token goes
  const int r = warp_last_le(a.q_off, a.n_req, x);
  int ctx, q0, T;
  if (r < 0 || r >= a.n_req || !rope_request(a, r, ctx, q0, T) || x - q0 >= T) return;
  const int p = ctx + x - q0;
  const int pos = a.pos ? a.pos[x] : p;
  if (pos < 0 || pos >= a.n_pos) {
    if (lane == 0) record_error(a.status, KVC_ERR_BOUNDS);
    return;
  }
  const int page = p / a.BS;
  const int32_t blk = a.block_table[(int64_t)r * a.max_blocks + page];
  int64_t slot = -1;
  if (blk >= 0 && blk < a.n_slots / a.BS) slot = (int64_t)blk * a.BS + (p - page * a.BS);
  else if (lane == 0) record_error(a.status, KVC_ERR_BOUNDS);
  // (pairs of columns: two products or sums an instruction)
  uint64_t cs[4], sn[4];
  {
    const float4 *t = reinterpret_cast<const float4 *>(a.tab + ((int64_t)pos * HALF + 8 * c) * 2);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float4 f = __ldg(t + e);
      cs[e] = pk2(f.x, f.z);
      sn[e] = pk2(f.y, f.w);
    }
  }
  const uint64_t minus = pk2(-1.f, -1.f);

  for (int g = g0; g < g1; g += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      const int hh = (g + u) * HPW + sub;
      const bool live = g + u < g1 && hh < heads;
      const int kind = hh < a.Hq ? 0 : hh < a.Hq + a.H ? 1 : 2;
      const uint32_t wl[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w};
      const uint32_t wh[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w};
      const uint4 vlo = lo[u], vhi = hi[u];
      uint64_t xl[4], xh[4], sq = 0;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        xl[e] = pk2(bf16_lo(wl[e]), bf16_hi(wl[e]));
        xh[e] = pk2(bf16_lo(wh[e]), bf16_hi(wh[e]));
      }
      if (g + kAhead < g1) load(u, g + kAhead + u);
#pragma unroll
      for (int e = 0; e < 4; e++) sq = fma2(xl[e], xl[e], fma2(xh[e], xh[e], sq));
      float sum, sum1;
      upk2(sq, sum, sum1);
      sum += sum1;
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (!live) continue;
      if (kind == 2) {
        if (slot >= 0) {
          uint16_t *d = a.vpool + (slot * a.H + hh - a.Hq - a.H) * D + 8 * c;
          *reinterpret_cast<uint4 *>(d) = vlo;
          *reinterpret_cast<uint4 *>(d + HALF) = vhi;
        }
        continue;
      }
      const uint16_t *w = kind ? a.wk : a.wq;
      if (w) {
        const float f = rsqrtf(sum * (1.f / D) + a.eps);
        const uint4 w0 = __ldg(reinterpret_cast<const uint4 *>(w + 8 * c));
        const uint4 w1 = __ldg(reinterpret_cast<const uint4 *>(w + HALF + 8 * c));
        const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
        const uint64_t f2 = pk2(f, f);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          xl[e] = mul2(mul2(xl[e], f2), pk2(bf16_lo(a0[e]), bf16_hi(a0[e])));
          xh[e] = mul2(mul2(xh[e], f2), pk2(bf16_lo(a1[e]), bf16_hi(a1[e])));
        }
      }
      if (kind == 1 && a.k_raw) {
        uint16_t *d = a.k_raw + (hh - a.Hq) * a.raw_stride + (int64_t)x * D + 8 * c;
        *reinterpret_cast<uint4 *>(d) = make_uint4(pack2(xl[0]), pack2(xl[1]), pack2(xl[2]), pack2(xl[3]));
        *reinterpret_cast<uint4 *>(d + HALF) = make_uint4(pack2(xh[0]), pack2(xh[1]), pack2(xh[2]), pack2(xh[3]));
      }
      uint32_t ol[4], oh[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        ol[e] = pack2(fma2(xl[e], cs[e], mul2(mul2(xh[e], minus), sn[e])));
        oh[e] = pack2(fma2(xh[e], cs[e], mul2(xl[e], sn[e])));
      }
      uint16_t *d;
      if (kind == 0) d = a.q_out + ((int64_t)x * a.Hq + hh) * D;
      else if (slot >= 0) d = a.kpool + (slot * a.H + hh - a.Hq) * D;
      else continue;
      *reinterpret_cast<uint4 *>(d + 8 * c) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
      *reinterpret_cast<uint4 *>(d + HALF + 8 * c) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
    }
  }
}

}  // namespace

cudaError_t launch_qkv_rope(const uint16_t *q, int64_t qs, const uint16_t *k, int64_t ks,
                            const uint16_t *v, int64_t vs, int n_tok, const uint16_t *wq,
                            const uint16_t *wk, float eps, const float *tab, int n_pos,
                            const int32_t *pos, const int32_t *q_off, const int32_t *ctx_len,
                            int n_req, const int32_t *block_table, int max_blocks,
                            uint16_t *kpool, uint16_t *vpool, int64_t n_slots, int H, int Hq,
                            int D, int BS, uint16_t *q_out, uint16_t *k_raw, int64_t raw_stride,
                            int32_t *status, cudaStream_t s) {
  RopeArgs a{};
  a.q = q, a.k = k, a.v = v, a.wq = wq, a.wk = wk, a.tab = tab;
  a.pos = pos, a.q_off = q_off, a.ctx_len = ctx_len, a.block_table = block_table;
  a.q_out = q_out, a.kpool = kpool, a.vpool = vpool, a.k_raw = k_raw, a.status = status;
  a.qs = qs, a.ks = ks, a.vs = vs, a.raw_stride = raw_stride, a.n_slots = n_slots;
  a.eps = eps;
  a.n_tok = n_tok, a.n_pos = n_pos, a.n_req = n_req, a.max_blocks = max_blocks;
  a.H = H, a.Hq = Hq, a.BS = BS;
  const int groups = (Hq + 2 * H + 512 / D - 1) / (512 / D);
  // parts of a token's heads: up to one group of heads each, while the GPU has room
  // for all the warps at once.  48 heads, D 128: one token 7.5 us in one part and 3.3 in
  // twelve; 512 tokens 7.9 in one, 5.2 in eight; 2048 11.4 in one, 9.9 in two, 11.6 in
  // four; 4096 17.4 in one and 18.6 in two.
  const int64_t room = kRopeWarps * kRopeCtas * (int64_t)device_sm_count();
  int parts = 1;
  while (parts < groups && 2 * (int64_t)n_tok * parts <= room) parts *= 2;
  const dim3 grid((unsigned)((n_tok + kRopeWarps - 1) / kRopeWarps),
                  (unsigned)(parts < groups ? parts : groups));
  if (D == 128) k_qkv_rope<128><<<grid, kRopeWarps * 32, 0, s>>>(a);
  else k_qkv_rope<64><<<grid, kRopeWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
