// q8_attn.cu — attention of a few rows per request over a history held in 8 bits
// and the bf16 rows behind it, one layer.  Row i of request r sees the len8
// positions of the history, the c positions of the bf16 cache and the nodes its
// mask marks:
//   z_p = scale·s_k·(q·k8_p) (history), scale·q·k_p (the others)
//   lse = ln Σ_p exp z_p,  out = Σ_p exp(z_p − lse)·v_p,  v_p = s_v·v8_p in the history
// with s_k and s_v the scales of the position's block and head.
//
// The unit of work, the split and the join are k_tree_rows' (tree_rows.cuh): a
// unit's tiles are those of its history and then those of its bf16 rows.  The
// bound is the stream: 2·D bytes per position of the history.
//
// e4m3 is a subset of fp16, so a byte becomes an fp16 operand by one conversion of
// two and the products are exact; q, a bf16 value, is exact in fp16 once each row
// is shifted by a power of two that puts its largest value just below 2^15 (what
// falls below fp16's range is 2^-39 of that value).  The scales stay out of the
// operands: a logit is multiplied by s_k, and the weight of V is
// 2^(z + log2 s_v − reference), on a running maximum of its own, so that no scale
// takes it out of fp16's range; the softmax's sum has its own exponent.
#include <float.h>

#include <algorithm>

#include "tree_rows.cuh"

namespace kvc {
namespace {

constexpr int kQ8Warps = 4;
constexpr int kQ8Threads = kQ8Warps * 32;
constexpr int kQ8Stages = 3;
constexpr int kQ8Stage = 8192;  // bytes of one warp's stage: K rows, then V rows
constexpr int kQ8Keys = 32;     // positions of a warp's stage of the history

struct Q8Args : TreeArgs {
  const uint8_t *k8, *v8;
  const float *kscale, *vscale;
  const int32_t *table8, *len8;
  int64_t n_blocks8;
  int max_blocks8;
};

// Request r's sizes; false when they are out of range.
__device__ __forceinline__ bool q8_request(const Q8Args &a, int r, int &n, int &c, int &q0, int &T) {
  n = a.len8[r];
  return tree_request(a, r, c, q0, T) && n >= 0 && n <= (int64_t)a.max_blocks8 * a.BS;
}
__device__ __forceinline__ int q8_tiles(int n) {
  return (n + kQ8Warps * kQ8Keys - 1) / (kQ8Warps * kQ8Keys);
}
// Row tiles and key tiles of request r (0 row tiles: nothing to do).
__device__ __forceinline__ void tree_tiles(const Q8Args &a, int r, int &n_rt, int &n_kt) {
  int n, c, q0, T;
  n_rt = n_kt = 0;
  if (!q8_request(a, r, n, c, q0, T)) return;
  n_rt = (T * a.G + a.rstep - 1) / a.rstep;
  n_kt = q8_tiles(n) + (c + T + a.tile - 1) / a.tile;
}

template <int D, int MT>
struct Q8Smem {
  static constexpr int kRing = kQ8Warps * kQ8Stages * kQ8Stage;
  static constexpr int kQh = kRing;                      // MT·16 rows of q in fp16, in the products' order
  static constexpr int kScale = kQh + MT * 16 * D * 2;   // (s_k, s_v) of a stage's positions
  static constexpr int kRow = kScale + kQ8Warps * kQ8Stages * kQ8Keys * 8;  // a row's power of two
  static constexpr int kValid = kRow + MT * 16 * 4;      // valid positions per (warp, stage)
  static constexpr int kMl = kValid + (kQ8Warps * kQ8Stages * 4 + 15) / 16 * 16;  // (max, sum) per (warp, row)
  static constexpr int kBytes = kMl + kQ8Warps * MT * 16 * 8;
  static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs fit an SM");
  static_assert(kQ8Warps * MT * 16 * D * 4 <= kRing, "the warps' O fit the ring");
  static_assert(2 * kQ8Keys * D <= kQ8Stage, "a stage of the history fits");
};

// Byte offset of 16-byte chunk c of 8-bit row `row`: eight rows of one chunk, and two
// rows of four chunks, hit distinct banks.
template <int D>
__device__ __forceinline__ uint32_t swz8(int row, int c) {
  const int f = D == 128 ? ((row & 1) << 2) | ((row >> 1) & 3) : (row >> 1) & 3;
  return (uint32_t)(row * D + ((c ^ f) << 4));
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t *w) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
// Two e4m3 (low and high byte of x) as fp16.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t x) {
  uint32_t d;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t x) {
  uint32_t d;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {  // a in the low half
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}
__device__ __forceinline__ void mma16816h(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, int MT>
__global__ void __launch_bounds__(kQ8Threads, 2)
k_q8_rows(Q8Args a) {
  using S = Q8Smem<D, MT>;
  constexpr int KT = 2048 / D, KS = D / 16, NT = D / 8, CH = D / 8, CH8 = D / 16;
  constexpr int R = MT * 16;
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 3;
  const uint32_t ring = smem_u32(sm) + warp * kQ8Stages * kQ8Stage;
  uint32_t *valid_s = reinterpret_cast<uint32_t *>(sm + S::kValid) + warp * kQ8Stages;
  const float2 *scale_s = reinterpret_cast<const float2 *>(sm + S::kScale) + warp * kQ8Stages * kQ8Keys;
  const uint32_t qhbase = smem_u32(sm + S::kQh);
  float *row_s = reinterpret_cast<float *>(sm + S::kRow);
  float2 *ml_s = reinterpret_cast<float2 *>(sm + S::kMl);

  asm volatile("griddepcontrol.launch_dependents;");
  if (blockIdx.x == 0)  // one report per bad request
    for (int r = tid; r < a.n_req; r += kQ8Threads) {
      int n, c, q0, T;
      if (!q8_request(a, r, n, c, q0, T)) record_error(a.status, KVC_ERR_BOUNDS);
    }
  auto tiles = [&](int x) {
    int n_rt, n_kt;
    tree_tiles(a, x, n_rt, n_kt);
    return (int64_t)a.H * n_rt * n_kt;
  };
  const WarpSums sums = warp_sums(a.n_req, tiles);
  const int64_t total = sums.total;
  const int n_cta = (int)min((int64_t)a.n_cta, total);  // every run holds a tile
  if ((int)blockIdx.x >= n_cta) return;
  const int64_t run0 = run_start(total, n_cta, blockIdx.x);
  const int64_t run1 = run_start(total, n_cta, blockIdx.x + 1);
  int64_t g = run0, before;  // next tile of the run
  int r, n8, c, q0, T, n_rt, n_kt;
  warp_find(sums, a.n_req, run0, tiles, r, before);
  q8_request(a, r, n8, c, q0, T);
  tree_tiles(a, r, n_rt, n_kt);
  int unit = (int)div64(g - before, n_kt);  // h·n_rt + row tile
  int t0 = (int)(g - before - (int64_t)unit * n_kt);

  const int64_t n_blocks = a.n_slots / a.BS;
  while (g < run1) {
    const int h = unit / n_rt, rt = unit % n_rt;
    const int t1 = (int)min((int64_t)n_kt, t0 + (run1 - g));
    const int th = q8_tiles(n8);  // tiles of the history
    const int n_rows = min(a.rstep, T * a.G - rt * a.rstep);
    const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
    const int32_t *bt8 = a.table8 + (int64_t)r * a.max_blocks8;
    const int end = c + T;

    // issue one stage: this warp's positions of tile t
    auto issue = [&](int t, int st) {
      const uint32_t dst = ring + st * kQ8Stage;
      if (t < th) {
        const int p = t * (kQ8Warps * kQ8Keys) + warp * kQ8Keys + lane;
        int32_t blk = -1, at = 0;
        if (p < n8) {
          const int pg = page_of(p, a.bs_inv);
          blk = bt8[pg];
          at = p - pg * a.BS;
          if (blk < 0 || blk >= a.n_blocks8) {
            record_error(a.status, KVC_ERR_BOUNDS);
            blk = -1;
          }
        }
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, blk >= 0);
        if (lane == 0) valid_s[st] = ok;
        const int64_t unit8 = (int64_t)max(blk, 0) * a.H + h;
        const uint32_t sc = smem_u32(sm + S::kScale) + ((warp * kQ8Stages + st) * kQ8Keys + lane) * 8;
        cp_async4(sc, a.kscale + unit8, blk >= 0);
        cp_async4(sc + 4, a.vscale + unit8, blk >= 0);
        constexpr int RPI = 32 / CH8;  // rows one instruction of the warp copies
        const int col = lane % CH8;
#pragma unroll
        for (int i = 0; i < kQ8Keys / RPI; i++) {
          const int row = i * RPI + lane / CH8;
          const int32_t b = __shfl_sync(0xFFFFFFFFu, blk, row), o = __shfl_sync(0xFFFFFFFFu, at, row);
          const int64_t from = (((int64_t)max(b, 0) * a.H + h) * a.BS + o) * D + col * 16;
          cp_async16(dst + swz8<D>(row, col), a.k8 + from, b >= 0);
          cp_async16(dst + kQ8Keys * D + swz8<D>(row, col), a.v8 + from, b >= 0);
        }
      } else {
        const int p0 = (t - th) * a.tile + warp * KT;
        int32_t slot = -1;
        if (lane < KT && p0 + lane < end) {
          const int p = p0 + lane;
          const int32_t b = bt[page_of(p, a.bs_inv)];
          if (b >= 0 && b < n_blocks) slot = b * a.BS + p - page_of(p, a.bs_inv) * a.BS;
          else record_error(a.status, KVC_ERR_BOUNDS);
        }
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, slot >= 0);
        if (lane == 0) valid_s[st] = ok;
        constexpr int RPI = 32 / CH;
        const int col = lane % CH;
#pragma unroll
        for (int i = 0; i < KT / RPI; i++) {
          const int row = i * RPI + lane / CH;
          const int32_t sl = __shfl_sync(0xFFFFFFFFu, slot, row);
          const int64_t from = ((int64_t)max(sl, 0) * a.H + h) * D + col * 8;
          cp_async16(dst + swz<D>(row, col), a.kpool + from, sl >= 0);
          cp_async16(dst + KT * D * 2 + swz<D>(row, col), a.vpool + from, sl >= 0);
        }
      }
    };
    const int n_t = t1 - t0;
#pragma unroll
    for (int s = 0; s < kQ8Stages - 1; s++) {
      if (s < n_t) issue(t0 + s, s);
      cp_commit();
    }
    // the row tile's queries in fp16 under the row's power of two (the bf16 rows' products
    // read them from memory)
    for (int e = tid; e < R * CH; e += kQ8Threads) {
      const int row = e / CH, col = e % CH, x = rt * a.rstep + row;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < n_rows)
        v = *reinterpret_cast<const uint4 *>(
            a.q + ((int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G) * D + col * 8);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < 4; u++) top = max(top, max(w[u] & 0x7FFFu, (w[u] >> 16) & 0x7FFFu));
#pragma unroll
      for (int o = 1; o < CH; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const int ex = max((int)(top >> 7) - 127 - 14, -126);
      if (col == 0) row_s[row] = __uint_as_float((uint32_t)(ex + 127) << 23);
      const float f = __uint_as_float((uint32_t)(127 - ex) << 23);
      // Dimension d = 64·hi + 16·j + 4·k + 2·b + e of a row is number 16·(4·hi + k) + 8·b +
      // 2·j + e of the products' order: thread j of a quad reads 16 bytes of K from 16·j on
      // (and from 64 + 16·j on), four of which are its values of one product.
      const int j = (col % 8) / 2, ks = 4 * (col / 8) + 2 * (col & 1);
#pragma unroll
      for (int u = 0; u < 4; u++)
        *reinterpret_cast<uint32_t *>(sm + S::kQh + swz<D>(row, 2 * (ks + u / 2) + (u & 1)) + 4 * j) =
            pack_f16x2(bf16_lo(w[u]) * f, bf16_hi(w[u]) * f);
    }
    __syncthreads();
    // one row tile of 16 keeps q in registers, in fp16 until the bf16 rows begin
    uint32_t qf[MT == 1 ? KS : 1][4];
    auto query16 = [&](int mt, int ks, uint32_t (&f)[4]) {  // a fragment of the bf16 queries
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        const int row = mt * 16 + hf * 8 + lane / 4, x = rt * a.rstep + row;
        const uint16_t *p = a.q + ((int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G) * D + 16 * ks + 2 * quad;
        f[hf] = row < n_rows ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
        f[2 + hf] = row < n_rows ? __ldg(reinterpret_cast<const uint32_t *>(p + 8)) : 0u;
      }
    };
    auto queries = [&](bool eight) {
      if (MT == 1)
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          if (eight) ldsm4(qhbase + swz<D>(lane % 16, 2 * ks + lane / 16), qf[MT == 1 ? ks : 0]);
          else query16(0, ks, qf[MT == 1 ? ks : 0]);
        }
    };
    bool hist = t0 < th;  // O's columns lie as the history's products leave them
    queries(hist);

    // m: largest logit, l: sum of the weights on it; mo: O's reference
    float o[MT][NT][4], m[MT][2], l[MT][2], mo[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      m[mt][0] = m[mt][1] = mo[mt][0] = mo[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; n++) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    }
    // The running maxima take in one row's new ones; O is rescaled.
    auto raise = [&](int mt, int hf, float mx, float mv, float &base, float &baseo) {
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      mv = fmaxf(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, 1));
      mv = fmaxf(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, 2));
      base = mx == -INFINITY ? 0.f : mx;
      baseo = mv == -INFINITY ? 0.f : mv;
      l[mt][hf] *= ex2(m[mt][hf] - base);
      const float f = ex2(mo[mt][hf] - baseo);
      m[mt][hf] = mx;
      mo[mt][hf] = mv;
      if (!__all_sync(0xFFFFFFFFu, f == 1.f))
#pragma unroll
        for (int n = 0; n < NT; n++) {
          o[mt][n][hf * 2] *= f;
          o[mt][n][hf * 2 + 1] *= f;
        }
    };
    // From the columns of the history's products (thread j of a quad: 16c + 4j + {0, 2} in
    // tile 2c, + {1, 3} in tile 2c + 1) to the usual ones (8n + 2j + {0, 1}).
    auto usual = [&]() {
      const int base = (lane & ~3) | (quad >> 1);
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int cc = 0; cc < NT / 2; cc++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
            const float v[4] = {o[mt][2 * cc][hf * 2], o[mt][2 * cc + 1][hf * 2],
                                o[mt][2 * cc][hf * 2 + 1], o[mt][2 * cc + 1][hf * 2 + 1]};
            float x[4], y[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
              x[e] = __shfl_sync(0xFFFFFFFFu, v[e], base);
              y[e] = __shfl_sync(0xFFFFFFFFu, v[e], base + 2);
            }
            o[mt][2 * cc][hf * 2] = quad & 1 ? x[2] : x[0];
            o[mt][2 * cc][hf * 2 + 1] = quad & 1 ? x[3] : x[1];
            o[mt][2 * cc + 1][hf * 2] = quad & 1 ? y[2] : y[0];
            o[mt][2 * cc + 1][hf * 2 + 1] = quad & 1 ? y[3] : y[1];
          }
      hist = false;
    };

    int st = 0;
    for (int t = t0; t < t1; t++) {
      cp_wait<kQ8Stages - 2>();
      __syncwarp();  // the stage has landed, and every lane is done with the one before it
      const int nx = t + kQ8Stages - 1;
      if (nx < t1) issue(nx, (st + kQ8Stages - 1) % kQ8Stages);
      cp_commit();
      const uint32_t okb = valid_s[st];
      const uint32_t kb = ring + st * kQ8Stage;
      if (t < th) {
        const uint32_t vb = kb + kQ8Keys * D;
        constexpr int N8 = kQ8Keys / 8;
        float s[MT][N8][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int n = 0; n < N8; n++) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
        uint32_t kw[N8][KS];
#pragma unroll
        for (int n = 0; n < N8; n++)
#pragma unroll
          for (int hi = 0; hi < KS / 4; hi++)
            lds128(kb + swz8<D>(8 * n + lane / 4, 4 * hi + quad), kw[n] + 4 * hi);
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          uint32_t qa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            if (MT == 1) {
#pragma unroll
              for (int e = 0; e < 4; e++) qa[mt][e] = qf[MT == 1 ? ks : 0][e];
            } else {
              ldsm4(qhbase + swz<D>(mt * 16 + lane % 16, 2 * ks + lane / 16), qa[mt]);
            }
          }
#pragma unroll
          for (int n = 0; n < N8; n++) {
            const uint32_t b0 = e4m3x2_f16x2(kw[n][ks]), b1 = e4m3x2_f16x2_hi(kw[n][ks]);
#pragma unroll
            for (int mt = 0; mt < MT; mt++) mma16816h(s[mt][n], qa[mt], b0, b1);
          }
        }
        float kz[2 * N8], lv[2 * N8];  // scale·s_k·log2 e and log2 s_v of this thread's positions
#pragma unroll
        for (int n = 0; n < N8; n++) {
          const float4 f = *reinterpret_cast<const float4 *>(scale_s + st * kQ8Keys + 8 * n + 2 * quad);
          kz[2 * n] = f.x * a.zscale;
          lv[2 * n] = lg2(f.y);
          kz[2 * n + 1] = f.z * a.zscale;
          lv[2 * n + 1] = lg2(f.w);
        }
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
            const float rs = row_s[mt * 16 + hf * 8 + lane / 4];
            float mx = m[mt][hf], mv = mo[mt][hf];
#pragma unroll
            for (int n = 0; n < N8; n++)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                float z = s[mt][n][hf * 2 + e] * rs * kz[2 * n + e];
                if (!((okb >> (8 * n + 2 * quad + e)) & 1u)) z = -INFINITY;
                s[mt][n][hf * 2 + e] = z;
                mx = fmaxf(mx, z);
                mv = fmaxf(mv, z + lv[2 * n + e]);
              }
            float base, baseo, sum = 0.f;
            raise(mt, hf, mx, mv, base, baseo);
#pragma unroll
            for (int n = 0; n < N8; n++)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const float z = s[mt][n][hf * 2 + e];
                sum += ex2(z - base);
                s[mt][n][hf * 2 + e] = ex2(z + lv[2 * n + e] - baseo);
              }
            l[mt][hf] += sum;
          }
#pragma unroll
        for (int kk = 0; kk < kQ8Keys / 16; kk++) {
          uint32_t pa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            pa[mt][0] = pack_f16x2(s[mt][2 * kk][0], s[mt][2 * kk][1]);
            pa[mt][1] = pack_f16x2(s[mt][2 * kk][2], s[mt][2 * kk][3]);
            pa[mt][2] = pack_f16x2(s[mt][2 * kk + 1][0], s[mt][2 * kk + 1][1]);
            pa[mt][3] = pack_f16x2(s[mt][2 * kk + 1][2], s[mt][2 * kk + 1][3]);
          }
#pragma unroll
          for (int cc = 0; cc < CH8; cc += 2) {
            // two keys by two neighbouring columns a register; after the exchange of the
            // middle bytes its halves are the operands of the even and of the odd columns
            uint32_t b[4];
            ldsm4t(vb + swz8<D>(kk * 16 + (lane & 15), cc + (lane >> 4)), b);
#pragma unroll
            for (int u = 0; u < 4; u++) b[u] = __byte_perm(b[u], 0, 0x3120);
#pragma unroll
            for (int u = 0; u < 2; u++) {
              const uint32_t e0 = e4m3x2_f16x2(b[2 * u]), e1 = e4m3x2_f16x2(b[2 * u + 1]);
              const uint32_t o0 = e4m3x2_f16x2_hi(b[2 * u]), o1 = e4m3x2_f16x2_hi(b[2 * u + 1]);
#pragma unroll
              for (int mt = 0; mt < MT; mt++) {
                mma16816h(o[mt][2 * (cc + u)], pa[mt], e0, e1);
                mma16816h(o[mt][2 * (cc + u) + 1], pa[mt], o0, o1);
              }
            }
          }
        }
      } else {
        if (hist) {
          usual();
          queries(false);
        }
        const uint32_t vb = kb + KT * D * 2;
        const int p0 = (t - th) * a.tile + warp * KT;
        float s[MT][KT / 8][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int n = 0; n < KT / 8; n++) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          uint32_t qa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            if (MT == 1) {
#pragma unroll
              for (int e = 0; e < 4; e++) qa[mt][e] = qf[MT == 1 ? ks : 0][e];
            } else {
              query16(mt, ks, qa[mt]);
            }
          }
#pragma unroll
          for (int kk = 0; kk < KT / 16; kk++) {
            uint32_t b[4];
            ldsm4(kb + swz<D>(kk * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), b);
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
              mma16816(s[mt][2 * kk], qa[mt], b[0], b[1]);
              mma16816(s[mt][2 * kk + 1], qa[mt], b[2], b[3]);
            }
          }
        }
        const bool masked = p0 + KT > c || okb != (KT == 32 ? 0xFFFFFFFFu : (1u << (KT & 31)) - 1u);
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
            uint32_t vis = 0xFFFFFFFFu;
            if (masked) {  // warp-uniform
              const int x = rt * a.rstep + mt * 16 + hf * 8 + lane / 4;
              vis = x < T * a.G ? visible_bits<KT>(a, x / a.G, q0, c, T, p0) & okb : 0u;
            }
            float mx = m[mt][hf], mv = mo[mt][hf];
#pragma unroll
            for (int n = 0; n < KT / 8; n++)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                float z = s[mt][n][hf * 2 + e] * a.zscale;
                if (!((vis >> (n * 8 + 2 * quad + e)) & 1u)) z = -INFINITY;
                s[mt][n][hf * 2 + e] = z;
                mx = fmaxf(mx, z);
                mv = fmaxf(mv, z);
              }
            float base, baseo, sum = 0.f;
            raise(mt, hf, mx, mv, base, baseo);
#pragma unroll
            for (int n = 0; n < KT / 8; n++)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const float z = s[mt][n][hf * 2 + e];
                sum += ex2(z - base);
                s[mt][n][hf * 2 + e] = ex2(z - baseo);
              }
            l[mt][hf] += sum;
          }
        tile_values<D, MT, KT>(a, s, o, vb, okb, rt, q0, c, T, p0);
      }
      st = (st + 1) % kQ8Stages;
    }
    cp_wait<0>();
    if (hist) usual();
    __syncthreads();  // every warp is done with the ring: it takes the warps' O

    float *o_s = reinterpret_cast<float *>(sm) + warp * R * D;
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        float sum = l[mt][hf];
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
        // O on the sum's reference
        const float f = m[mt][hf] == -INFINITY || mo[mt][hf] == -INFINITY ? 1.f : ex2(mo[mt][hf] - m[mt][hf]);
        const int row = mt * 16 + hf * 8 + lane / 4;
        if (quad == 0) ml_s[warp * R + row] = make_float2(m[mt][hf], sum);
#pragma unroll
        for (int n = 0; n < NT; n++)
          *reinterpret_cast<float2 *>(o_s + row * D + ((n * 8 + 2 * quad) ^ ((row & 3) << 3))) =
              make_float2(o[mt][n][hf * 2] * f, o[mt][n][hf * 2 + 1] * f);
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == n_kt;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (g != run0);
    for (int e = tid; e < n_rows * (D / 4); e += kQ8Threads) {
      const int row = e / (D / 4), d4 = (e % (D / 4)) * 4;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kQ8Warps; w++) mx = fmaxf(mx, ml_s[w * R + row].x);
      const float base = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kQ8Warps; w++) {
        const float2 ml = ml_s[w * R + row];
        // (this warp saw nothing of the row; logits that are all NaN leave a NaN sum)
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        const float f = ex2(ml.x - base);
        sum = fmaf(ml.y, f, sum);
        const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sm) +
                                                           (w * R + row) * D + (d4 ^ ((row & 3) << 3)));
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        const int x = rt * a.rstep + row;
        const int64_t qr = (int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2 *>(a.out + qr * D + d4) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (d4 == 0) a.lse[qr] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
      } else {
        *reinterpret_cast<float4 *>(a.part_o + (slot * R + row) * D + d4) = acc;
        if (d4 == 0) a.part_ml[slot * R + row] = make_float2(mx, sum);
      }
    }
    g += n_t;
    t0 = 0;
    if (g < run1) {
      if (t1 == n_kt && ++unit == a.H * n_rt) {
        unit = 0;
        do {
          r++;
          tree_tiles(a, r, n_rt, n_kt);
        } while (n_rt == 0);  // g < run1 ≤ total: a later request holds tile g
        q8_request(a, r, n8, c, q0, T);
      }
      __syncthreads();
    }
  }
}

// Rows per tile and grid of a call.
void q8_plan(int n_req, int max_blocks8, int max_blocks, int max_tree, int H, int Hq, int D, int BS,
             int &rows, int &tile, int &n_cta, int &max_rt) {
  const int64_t R = (int64_t)max_tree * (Hq / H);
  rows = R <= 16 ? 16 : 32;
  tile = kQ8Warps * (2048 / D);
  max_rt = (int)((R + rows - 1) / rows);
  const int64_t kt = ((int64_t)max_blocks8 * BS + kQ8Warps * kQ8Keys - 1) / (kQ8Warps * kQ8Keys) +
                     ((int64_t)max_blocks * BS + tile - 1) / tile;
  n_cta = (int)std::min<int64_t>(2 * device_sm_count(), (int64_t)n_req * H * max_rt * kt);
}

template <int D, int MT>
cudaError_t launch_q8_rows(const Q8Args &a, cudaStream_t s) {
  constexpr int smem = Q8Smem<D, MT>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(k_q8_rows<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_q8_rows<D, MT><<<a.n_cta, kQ8Threads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t q8_attn_ws_bytes(int n_req, int max_blocks8, int max_blocks, int max_tree, int H, int Hq, int D,
                        int BS) {
  int rows, tile, n_cta, max_rt;
  q8_plan(n_req, max_blocks8, max_blocks, max_tree, H, Hq, D, BS, rows, tile, n_cta, max_rt);
  return (size_t)2 * n_cta * rows * (D * sizeof(float) + sizeof(float2));
}

cudaError_t launch_q8_attn(const uint16_t *q, const uint8_t *k8, const uint8_t *v8, const float *kscale,
                           const float *vscale, int64_t n_blocks8, const int32_t *table8,
                           int max_blocks8, const int32_t *len8, const uint16_t *kpool,
                           const uint16_t *vpool, int64_t n_slots, const int32_t *block_table,
                           int max_blocks, const int32_t *ctx_len, const int32_t *q_off,
                           const uint32_t *tree_mask, int mask_words, int n_req, int n_q, int max_tree,
                           int H, int Hq, int D, int BS, float scale, uint16_t *out, float *lse,
                           void *ws, int32_t *status, cudaStream_t s) {
  Q8Args a{};
  a.q = q, a.kpool = kpool, a.vpool = vpool, a.block_table = block_table;
  a.ctx_len = ctx_len, a.q_off = q_off, a.mask = tree_mask, a.out = out, a.lse = lse;
  a.status = status, a.n_slots = n_slots, a.max_blocks = max_blocks, a.mask_words = mask_words;
  a.n_req = n_req, a.n_q = n_q, a.max_tree = max_tree;
  a.H = H, a.Hq = Hq, a.G = Hq / H, a.BS = BS, a.bs_inv = page_inverse(BS);
  a.zscale = scale != 0.f ? scale * kLog2e : 1e-30f;  // (so that −inf stays −inf when scaled)
  a.k8 = k8, a.v8 = v8, a.kscale = kscale, a.vscale = vscale, a.table8 = table8, a.len8 = len8;
  a.n_blocks8 = n_blocks8, a.max_blocks8 = max_blocks8;
  int max_rt;
  q8_plan(n_req, max_blocks8, max_blocks, max_tree, H, Hq, D, BS, a.rows, a.tile, a.n_cta, max_rt);
  a.rstep = a.rows;
  a.part_o = reinterpret_cast<float *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)2 * a.n_cta * a.rows * D);
  const cudaError_t e = D == 128 ? (a.rows == 16 ? launch_q8_rows<128, 1>(a, s) : launch_q8_rows<128, 2>(a, s))
                                 : (a.rows == 16 ? launch_q8_rows<64, 1>(a, s) : launch_q8_rows<64, 2>(a, s));
  if (e != cudaSuccess) return e;
  return launch_join(a, D, max_rt, s);
}

}  // namespace kvc
