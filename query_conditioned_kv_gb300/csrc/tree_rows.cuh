// tree_rows.cuh — what the kernels share that give a few query rows of a request
// all of its keys (tree_attn.cu, q8_attn.cu): a call's arguments, how key tiles
// are dealt out to the CTAs, which keys a row sees, and the join of a unit's parts.
#pragma once

#include <math.h>

#include <type_traits>

#include "kvc_internal.cuh"
#include "mma_ptx.cuh"

namespace kvc {
namespace {

using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
  static constexpr bool kMeans = false;  // part_o holds sums, not means
  const uint16_t *q, *kpool, *vpool;
  const int32_t *block_table, *ctx_len, *q_off;
  const uint32_t *mask;  // [n_q][mask_words] or NULL (a chain)
  uint16_t *out;
  float *lse;
  int32_t *status;
  float2 *part_ml;  // [2·grid][rows]: (max in log2, sum) of a partial
  float *part_o;    // [2·grid][rows][D]
  int64_t n_slots;
  int max_blocks, mask_words, n_req, n_q, max_tree, H, Hq, G, BS;
  int rows;      // rows of a row tile's buffers
  int rstep;     // rows of a row tile (whole nodes where the tile holds several)
  int tile;      // keys per tile
  int n_cta;     // CTAs the tiles are dealt out to
  uint32_t bs_inv;  // ⌈2^32 / BS⌉ (0: BS = 1)
  float zscale;  // scale·log2(e)
  int join_rows;  // rows of a join CTA
};

// Request r's sizes; false when they are out of range.
__device__ __forceinline__ bool tree_request(const TreeArgs &a, int r, int &c, int &q0, int &T) {
  c = a.ctx_len[r];
  q0 = a.q_off[r];
  const int64_t t = (int64_t)a.q_off[r + 1] - q0;
  T = (int)t;
  return c >= 0 && q0 >= 0 && t >= 0 && t <= a.max_tree && q0 + t <= a.n_q &&
         c + t <= (int64_t)a.max_blocks * a.BS;
}

// Row tiles and key tiles of request r (0 row tiles: nothing to do).
__device__ __forceinline__ void tree_tiles(const TreeArgs &a, int r, int &n_rt, int &n_kt) {
  int c, q0, T;
  n_rt = n_kt = 0;
  if (!tree_request(a, r, c, q0, T)) return;
  n_rt = (T * a.G + a.rstep - 1) / a.rstep;
  n_kt = (c + T + a.tile - 1) / a.tile;
}

// How `total` tiles are dealt out: CTA c begins at ⌊total·c / n_cta⌋.
__device__ __forceinline__ int64_t run_start(int64_t total, int n_cta, int cta) {
  return div64(total * cta, n_cta);
}
// The CTA whose run holds tile t: the last c with total·c < (t + 1)·n_cta.
__device__ __forceinline__ int run_owner(int64_t total, int n_cta, int64_t t) {
  return (int)div64((t + 1) * n_cta - 1, total);
}

// Tiles of request r, all heads.
__device__ __forceinline__ int64_t request_tiles(const TreeArgs &a, int r) {
  int n_rt, n_kt;
  tree_tiles(a, r, n_rt, n_kt);
  return (int64_t)a.H * n_rt * n_kt;
}

// Bits k < KT of the keys p0 + k that row `i` (node) of the request sees.
template <int KT>
__device__ __forceinline__ uint32_t visible_bits(const TreeArgs &a, int i, int q0, int c, int T,
                                                 int p0) {
  constexpr uint32_t full = KT == 32 ? 0xFFFFFFFFu : (1u << (KT & 31)) - 1u;
  const int j0 = p0 - c;  // node index of the first key (negative: a cached position)
  if (j0 + KT <= 0) return full;
  uint32_t bits = 0;
  if (j0 < 0) bits = (1u << -j0) - 1u;  // −j0 < KT ≤ 32
  const int lo = max(j0, 0);
  if (lo >= T) return bits;
  uint32_t node;  // bits of the nodes lo … lo + 31
  if (a.mask) {
    const uint32_t *m = a.mask + (int64_t)(q0 + i) * a.mask_words;
    const int w = lo >> 5, s = lo & 31;
    uint64_t two = m[w];
    if (w + 1 < a.mask_words) two |= (uint64_t)m[w + 1] << 32;
    node = (uint32_t)(two >> s);
  } else {
    node = i < lo ? 0u : i - lo >= 31 ? 0xFFFFFFFFu : (2u << (i - lo)) - 1u;
  }
  if (T - lo < 32) node &= (1u << (T - lo)) - 1u;
  bits |= j0 < 0 ? node << -j0 : node;
  return bits & full;
}

// The factor under which a part's O, v, joins a row: a share below fp32 is not 0, and an
// infinity stays one under it.
__device__ __forceinline__ float share_of(float v, float f) {
  return f == 0.f && fabsf(v) == INFINITY ? 1.f : f;
}

// Joins the partials of one (request, KV head, row tile) that was split over
// CTAs: blockIdx.x = (request, KV head), blockIdx.y = row tile, blockIdx.z a
// group of rows.  W warps share a row's partials (W 4: warp w takes the parts w,
// w + 4, …, all in flight at once; their results are added in order), or each
// takes join_rows / 4 rows of its own (W 1).  Bound by latency, so the fewest
// dependent loads: sizes, then maxima and sums, then O.  Where the parts are means of
// the values (O over the part's sum: Args::kMeans), so is what is joined at every step.
template <class Args, int D, int W>
__global__ void __launch_bounds__(128)
k_tree_join(Args a) {
  constexpr int E = D / 32;
  __shared__ float sh_o[W][D];
  __shared__ float2 sh_ml[W];
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, rt = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t before = 0, total = 0;
  int n_rt = 0, n_kt = 0;
#pragma unroll 2
  for (int x0 = 0; x0 < a.n_req; x0 += 32) {  // (every warp for itself)
    const int x = x0 + lane;
    int rt_x = 0, kt_x = 0;
    if (x < a.n_req) tree_tiles(a, x, rt_x, kt_x);
    const int64_t n = (int64_t)a.H * rt_x * kt_x;
    total += n;
    if (x < r) before += n;
    if (x0 <= r && r < x0 + 32) {
      n_rt = __shfl_sync(0xFFFFFFFFu, rt_x, r - x0);
      n_kt = __shfl_sync(0xFFFFFFFFu, kt_x, r - x0);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  }
  const int q0 = a.q_off[r], T = a.q_off[r + 1] - q0;
  // in every CTA: the grid may not end before the kernel whose partials it joins
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (rt >= n_rt) return;
  const int64_t g0 = before + ((int64_t)h * n_rt + rt) * n_kt;
  const int n_cta = (int)min((int64_t)a.n_cta, total);
  const int c0 = run_owner(total, n_cta, g0), c1 = run_owner(total, n_cta, g0 + n_kt - 1);
  if (c0 == c1) return;  // written whole
  const int64_t first = 2 * (int64_t)c0 + (run_start(total, n_cta, c0) != g0);
  const int n_part = c1 - c0 + 1;
  const int n_rows = min(a.rstep, T * a.G - rt * a.rstep), d0 = lane * E;
  const int row0 = W == 1 ? blockIdx.z * a.join_rows + warp : blockIdx.z;
  const int row1 = W == 1 ? min(n_rows, (int)(blockIdx.z + 1) * a.join_rows) : min(n_rows, row0 + 1);
  for (int row = row0; row < row1; row += 4) {
    float mx, sum, acc[E];
    auto gather = [&](auto Inf) {  // Inf: a part may hold an infinity of no share
      mx = -INFINITY;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; e++) acc[e] = 0.f;
      for (int i0 = W == 1 ? 0 : warp; i0 < n_part; i0 += 32 * W) {
        // part i is slot first (i = 0) or 2·(c0 + i): later CTAs begin inside the unit
        const int mine = i0 + W * lane;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (mine < n_part)
          ml = a.part_ml[(mine == 0 ? first : 2 * (int64_t)(c0 + mine)) * a.rows + row];
        float m = ml.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float now = fmaxf(mx, m), base = now == -INFINITY ? 0.f : now;
        const float keep = mx == -INFINITY ? 0.f : ex2(mx - base);
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - base);
        float s = ml.y * f;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        float keep_o = keep * sum, fo = f * ml.y;  // a part's share of O
        sum = fmaf(sum, keep, s);
        if constexpr (Args::kMeans) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          keep_o *= inv;
          fo *= inv;
        } else {
          keep_o = keep;
          fo = f;
        }
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] *= Inf.value ? share_of(acc[e], keep_o) : keep_o;
        mx = now;
        const int n = min(32, (n_part - i0 + W - 1) / W);
#pragma unroll 8
        for (int k = 0; k < n; k++) {
          const int i = i0 + W * k;
          const float *o = a.part_o + ((i == 0 ? first : 2 * (int64_t)(c0 + i)) * a.rows + row) * D + d0;
          const float fk = __shfl_sync(0xFFFFFFFFu, fo, k);
          float v[E];
          if constexpr (E == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(o);
          else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(o);
#pragma unroll
          for (int e = 0; e < E; e++) acc[e] = fmaf(v[e], Inf.value ? share_of(v[e], fk) : fk, acc[e]);
        }
      }
    };
    gather(std::false_type());
    if constexpr (Args::kMeans) {  // (0·inf is NaN: only then looked at)
      bool nan = false;
#pragma unroll
      for (int e = 0; e < E; e++) nan |= isnan(acc[e]);
      if (__any_sync(0xFFFFFFFFu, nan)) gather(std::true_type());
    }
    if constexpr (W > 1) {
#pragma unroll
      for (int e = 0; e < E; e++) sh_o[warp][d0 + e] = acc[e];
      if (lane == 0) sh_ml[warp] = make_float2(mx, sum);
      __syncthreads();
      if (warp != 0) return;
      mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; w++) mx = fmaxf(mx, sh_ml[w].x);
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; e++) acc[e] = 0.f;
#pragma unroll
      for (int w = 0; w < W; w++)
        sum = fmaf(sh_ml[w].y, sh_ml[w].x == -INFINITY ? 0.f : ex2(sh_ml[w].x - mx), sum);
      const float inv = !Args::kMeans ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int w = 0; w < W; w++) {
        float f = sh_ml[w].x == -INFINITY ? 0.f : ex2(sh_ml[w].x - mx);
        if constexpr (Args::kMeans) f *= sh_ml[w].y * inv;
#pragma unroll
        for (int e = 0; e < E; e++) {
          const float v = sh_o[w][d0 + e];
          acc[e] = fmaf(v, Args::kMeans ? share_of(v, f) : f, acc[e]);
        }
      }
    }
    const float inv = Args::kMeans ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
    const int x = rt * a.rstep + row;
    const int64_t qr = (int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; e++) w[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if constexpr (E == 4) *reinterpret_cast<uint2 *>(a.out + qr * D + d0) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(a.out + qr * D + d0) = w[0];
    if (d0 == 0) a.lse[qr] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
  }
}

// The join's launch, after the kernel that wrote the parts.
template <class Args>
cudaError_t launch_join(Args a, int D, int max_rt, cudaStream_t s) {
  // four warps a row where a unit is cut into many parts
  const bool many = a.n_cta >= 6 * (int64_t)a.n_req * a.H * max_rt;
  auto *join = D == 128 ? (many ? k_tree_join<Args, 128, 4> : k_tree_join<Args, 128, 1>)
                        : (many ? k_tree_join<Args, 64, 4> : k_tree_join<Args, 64, 1>);
  // as many CTAs as the GPU holds at once, so that no warp's rows wait for one another
  a.join_rows = many ? 1 : 4;
  while (!many && a.join_rows < a.rstep &&
         (int64_t)a.n_req * a.H * max_rt * a.rstep > (int64_t)a.join_rows * 16 * device_sm_count())
    a.join_rows *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.n_req * a.H), (unsigned)max_rt,
                     (unsigned)((a.rstep + a.join_rows - 1) / a.join_rows));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join, a);
}

}  // namespace
}  // namespace kvc
