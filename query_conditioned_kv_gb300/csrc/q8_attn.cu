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
// k_q8_rows: each of a CTA's four warps streams its own quarter of every tile (32
// positions of the history, or 4 KB of bf16 keys) through a private ring of shared memory,
// by TMA boxes of rows of a block where every position of the quarter is there, else by
// cp.async; no barrier until the run ends.  Positions are the products' M dimension
//   Sᵀ[position][row] = K·Qᵀ,   Oᵀ[d][row] += Vᵀ·Pᵀ
// (mma.sync m16n8k16), so that rows come in eights and a token of four heads does not pay
// for sixteen rows: 64 products a quarter tile and eight rows, half of what rows as M take.
// e4m3 is a subset of fp16, so a byte becomes an fp16 operand by a conversion of two and
// the products are exact.  q, bf16 values of 8 bits, becomes fp16 under a power of two per
// row that puts its largest value into [2^14, 2^15): exact while a value's last bit is 2^-24
// or more (from 2^-31 of the largest on), below that rounded by up to 2^-25 (2^-39 of it).
// V's operand is read by the transposing ldmatrix, two bytes a number: a register then holds
// two columns of two positions, and O's columns come in pairs until usual() puts them in order.
//
// The scales stay out of the operands: a logit is multiplied by s_k, and P is the weight
// times s_v on a reference of its own.  References are a row's largest over its first
// tile (less kQ8Room, in log2), raised when a weight passes 2^15: weights fit fp16 whatever the
// scales, and a tile needs no maximum.
//
// What leaves a warp is the mean of its values, and every join adds means by their shares
// (sums on the softmax's reference would pass fp32 where |v| passes 2^113).  Infinite values of
// nodes stay out of the products and are added to the means; an infinity under a share that
// fp32 loses is looked for where a join gives NaN.
//
// One token, 8 KV and 32 query heads, D 128: 64 requests of up to 8192 142 us, 5.9 TB/s, 87 % of
// a copy's rate; one of 4096 13, latency.  18 rows per KV head over two requests of 131072 129
// us, 4.2 TB/s, bound by products and conversions (125 with sums for means and infinities in the
// products).  Rows as the products' M took 166 and 179.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "tree_rows.cuh"

namespace kvc {
namespace {

constexpr int kQ8Warps = 4;
constexpr int kQ8Threads = kQ8Warps * 32;
// CTAs per SM and stages of a warp's ring, by the row tile's eights of rows.  Of 8 rows, 64
// requests of up to 8192: three CTAs 139 us, two 142.  Of 24 rows, two of 131072: two 122, three,
// which spill, 184.
constexpr int q8_ctas(int nr) { return nr <= 2 ? 3 : 2; }
constexpr int q8_stages(int nr) { return nr <= 2 ? 2 : 3; }
constexpr int kQ8Stage = 8192;  // bytes of one warp's stage: K rows, then V rows
constexpr int kQ8Keys = 32;     // positions of a warp's stage of the history
constexpr float kQ8Unset = -FLT_MAX;   // reference of a row that has seen nothing
constexpr float kQ8Room = 8.f;         // log2 of the largest weight of a row's first tile
constexpr float kQ8Most = 32768.f;     // weight, and sum of a thread's four, that raises the references
constexpr float kQ8Round = 1048576.f;  // |reference| from which logits are rounded before the difference

struct Q8Args : TreeArgs {
  static constexpr bool kMeans = true;  // a sum of values times 2^8 to 2^15 may pass fp32
  const uint8_t *k8, *v8;
  const float *kscale, *vscale;
  const int32_t *table8, *len8;
  int64_t n_blocks8;
  int max_blocks8;
  int box8;  // rows of a TMA box of the 8-bit pools (a divisor of the page size), 0: no TMA
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

template <int D, int NR>
struct Q8Smem {
  static constexpr int R = 8 * NR, kQ8Stages = q8_stages(NR);
  static constexpr int kRing = kQ8Warps * kQ8Stages * kQ8Stage;
  static constexpr int kQh = kRing;              // the rows of q in fp16, in the products' order
  static constexpr int kScale = kQh + R * D * 2; // (s_k, s_v) of a stage's positions
  static constexpr int kRow = kScale + kQ8Warps * kQ8Stages * kQ8Keys * 8;  // a row's power of two
  static constexpr int kValid = kRow + R * 4;    // valid positions per (warp, stage)
  static constexpr int kMl = kValid + (kQ8Warps * kQ8Stages * 4 + 15) / 16 * 16;  // (reference, sum) per (warp, row)
  static constexpr int kClMl = kMl + kQ8Warps * R * 8;   // (reference, sum) of the CTA, per row
  static constexpr int kFull = kClMl + R * 8;            // barriers per (warp, stage), then a word
  static constexpr int kBytes = kFull + kQ8Warps * kQ8Stages * 8 + 16;
  static_assert(q8_ctas(NR) * (kBytes + 1024) <= 228 * 1024, "the CTAs fit an SM");
  static constexpr int kClO = kQ8Warps * R * D * 4;      // the CTA's O, behind the warps'
  static_assert(kClO + R * D * 4 <= kRing, "the warps' and the CTA's O fit the ring");
  static_assert(2 * kQ8Keys * D <= kQ8Stage, "a stage of the history fits");
};

// Byte offset of 16-byte chunk c of 8-bit row `row`: the 128- and 64-byte swizzles of TMA.
template <int D>
__device__ __forceinline__ uint32_t swz8(int row, int c) {
  return (uint32_t)(row * D + ((c ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4));
}
__device__ __forceinline__ void tma_load_2d_if(uint32_t lead, uint32_t dst, const CUtensorMap *map, int x,
                                               int y, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n"
      " @q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(lead)
      : "memory");
}
// An 8×8 matrix of 16-bit values (row t/4, columns 2·(t%4) + {0, 1} in thread t), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
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
__device__ __forceinline__ void add_part(float4 &acc, const float4 &v, float f) {
  acc.x = fmaf(v.x, f, acc.x);
  acc.y = fmaf(v.y, f, acc.y);
  acc.z = fmaf(v.z, f, acc.z);
  acc.w = fmaf(v.w, f, acc.w);
}
__device__ __forceinline__ void add_part_inf(float4 &acc, const float4 &v, float f) {
  acc.x = fmaf(v.x, share_of(v.x, f), acc.x);
  acc.y = fmaf(v.y, share_of(v.y, f), acc.y);
  acc.z = fmaf(v.z, share_of(v.z, f), acc.z);
  acc.w = fmaf(v.w, share_of(v.w, f), acc.w);
}
__device__ __forceinline__ bool any_nan(const float4 &v) { return isnan(v.x) || isnan(v.y) || isnan(v.z) || isnan(v.w); }
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The values of nodes that are not finite, among a warp's keys of the tiles t0 … t1, to the
// rows of its means that see them.  (Apart: seldom called.)
template <int D, int KT>
__device__ __noinline__ void add_infinite(const Q8Args &a, float *o_s, const int32_t *bt, int t0, int t1,
                                          int th, int h, int rt, int n_rows, int q0, int c, int T) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n_blocks = a.n_slots / a.BS;
  __syncwarp();
  for (int t = max(t0, th); t < t1; t++) {
    const int p0 = (t - th) * a.tile + warp * KT;
    if (p0 + KT <= c) continue;  // (cached rows only: left to the products)
    for (int p = p0; p < min(p0 + KT, c + T); p++) {
      const int pg = page_of(p, a.bs_inv);
      const int32_t b = bt[pg];
      if (b < 0 || b >= n_blocks) continue;
      const uint16_t *vr = a.vpool + (((int64_t)b * a.BS + p - pg * a.BS) * a.H + h) * D;
      for (int d = lane; d < D; d += 32) {
        const float v = bf16_lo(vr[d]);
        if (fabsf(v) < INFINITY) continue;
        for (int row = 0; row < n_rows; row++)
          if ((visible_bits<KT>(a, (rt * a.rstep + row) / a.G, q0, c, T, p0) >> (p - p0)) & 1u)
            o_s[row * D + (d ^ (((row >> 1) & 3) << 3))] += v;
      }
    }
  }
}

// CL: a cluster takes a unit, each CTA a part of its tiles, and joins the parts from one
// another's shared memory.
template <int D, int NR, bool CL>
__global__ void __launch_bounds__(kQ8Threads, q8_ctas(NR))
k_q8_rows(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Q8Args a) {
  using S = Q8Smem<D, NR>;
  constexpr int KT = 2048 / D, KS = D / 16, CH = D / 8, CH8 = D / 16;
  constexpr int R = 8 * NR, kQ8Stages = S::kQ8Stages;
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 3, g8 = lane >> 2;
  const uint32_t ring = smem_u32(sm) + warp * kQ8Stages * kQ8Stage;
  uint32_t *valid_s = reinterpret_cast<uint32_t *>(sm + S::kValid) + warp * kQ8Stages;
  const float2 *scale_s = reinterpret_cast<const float2 *>(sm + S::kScale) + warp * kQ8Stages * kQ8Keys;
  const uint32_t qhbase = smem_u32(sm + S::kQh);
  const uint32_t full = smem_u32(sm + S::kFull) + warp * kQ8Stages * 8;
  volatile int *failed = reinterpret_cast<volatile int *>(sm + S::kFull + kQ8Warps * kQ8Stages * 8);
  float *row_s = reinterpret_cast<float *>(sm + S::kRow);
  float2 *ml_s = reinterpret_cast<float2 *>(sm + S::kMl);

  if (!CL) asm volatile("griddepcontrol.launch_dependents;");
  if (lane == 0) {
    for (int i = 0; i < kQ8Stages; i++) mbar_init(full + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 0) *failed = 0;
  int r, n8, c, q0, T, n_rt, n_kt, unit, t0;
  int64_t g, run0, run1;  // next tile of the run, its begin and end
  if constexpr (CL) {
    const int S = (int)cluster_nrank(), rank = (int)cluster_rank(), u = blockIdx.x / S;
    r = u / a.H;
    unit = u % a.H;
    const bool valid = q8_request(a, r, n8, c, q0, T);
    if (!valid && unit == 0 && rank == 0 && tid == 0) record_error(a.status, KVC_ERR_BOUNDS);
    tree_tiles(a, r, n_rt, n_kt);
    if (n_rt == 0) return;  // (the whole cluster)
    t0 = n_kt * rank / S;
    g = run0 = 0;
    run1 = n_kt * (rank + 1) / S - t0;
  } else {
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
    int64_t before;
    const int n_cta = (int)min((int64_t)a.n_cta, total);  // every run holds a tile
    if ((int)blockIdx.x >= n_cta) return;
    run0 = g = run_start(total, n_cta, blockIdx.x);
    run1 = run_start(total, n_cta, blockIdx.x + 1);
    warp_find(sums, a.n_req, run0, tiles, r, before);
    q8_request(a, r, n8, c, q0, T);
    tree_tiles(a, r, n_rt, n_kt);
    unit = (int)div64(g - before, n_kt);  // h·n_rt + row tile
    t0 = (int)(g - before - (int64_t)unit * n_kt);
  }
  __syncthreads();

  const int64_t n_blocks = a.n_slots / a.BS;
  uint32_t boxed = 0, phase = 0;  // bits of the stages: filled by TMA, the barrier's parity
  while (CL || g < run1) {
    const int h = unit / n_rt, rt = unit % n_rt;
    const int t1 = (int)min((int64_t)n_kt, t0 + (run1 - g));
    const int th = q8_tiles(n8);  // tiles of the history
    const int n_rows = min(a.rstep, T * a.G - rt * a.rstep);
    const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
    const int32_t *bt8 = a.table8 + (int64_t)r * a.max_blocks8;
    const int end = c + T;

    // the block id of this lane's position of tile t, looked up a tile ahead
    int32_t next_blk;
    auto look = [&](int t) {
      next_blk = -1;
      if (t < th) {
        const int p = (t * kQ8Warps + warp) * kQ8Keys + lane;
        if (p < n8) next_blk = bt8[page_of(p, a.bs_inv)];
      } else if (t < t1) {
        const int p = (t - th) * a.tile + warp * KT + lane;
        if (lane < KT && p < end) next_blk = bt[page_of(p, a.bs_inv)];
      }
    };
    // issue one stage: this warp's positions of tile t
    auto issue = [&](int t, int st) {
      const uint32_t dst = ring + st * kQ8Stage;
      int32_t blk = next_blk;
      look(t + 1);
      boxed &= ~(1u << st);
      if (t < th) {
        const int p = (t * kQ8Warps + warp) * kQ8Keys + lane;
        const int at = p - page_of(p, a.bs_inv) * a.BS;
        if (p < n8 && (blk < 0 || blk >= a.n_blocks8)) {
          record_error(a.status, KVC_ERR_BOUNDS);
          blk = -1;
        }
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, blk >= 0);
        if (lane == 0) valid_s[st] = ok;
        const int64_t unit8 = (int64_t)max(blk, 0) * a.H + h;
        const uint32_t sc = smem_u32(sm + S::kScale) + ((warp * kQ8Stages + st) * kQ8Keys + lane) * 8;
        cp_async4(sc, a.kscale + unit8, blk >= 0);
        cp_async4(sc + 4, a.vscale + unit8, blk >= 0);
        if (a.box8 && ok == 0xFFFFFFFFu) {
          const uint32_t bar = full + 8 * st;
          // (what was written and read here before is ordered before the copies)
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          if (lane == 0) mbar_expect_tx(bar, 2 * kQ8Keys * D);
          __syncwarp();
          boxed |= 1u << st;
          const int row = (int)unit8 * a.BS + at;
          for (int k = 0; k < kQ8Keys; k += a.box8) {
            const int y = __shfl_sync(0xFFFFFFFFu, row, k);
            tma_load_2d_if(lane == 0, dst + k * D, &tm_k, 0, y, bar);
            tma_load_2d_if(lane == 0, dst + (kQ8Keys + k) * D, &tm_v, 0, y, bar);
          }
        } else {
          constexpr int RPI = 32 / CH8;  // rows one instruction of the warp copies
          const int col = lane % CH8;
#pragma unroll 2
          for (int i = 0; i < kQ8Keys / RPI; i++) {
            const int row = i * RPI + lane / CH8;
            const int32_t b = __shfl_sync(0xFFFFFFFFu, blk, row), o = __shfl_sync(0xFFFFFFFFu, at, row);
            const int64_t from = (((int64_t)max(b, 0) * a.H + h) * a.BS + o) * D + col * 16;
            cp_async16(dst + swz8<D>(row, col), a.k8 + from, b >= 0);
            cp_async16(dst + kQ8Keys * D + swz8<D>(row, col), a.v8 + from, b >= 0);
          }
        }
      } else {
        const int p = (t - th) * a.tile + warp * KT + lane;
        int32_t slot = -1;
        if (lane < KT && p < end) {
          if (blk >= 0 && blk < n_blocks) slot = blk * a.BS + p - page_of(p, a.bs_inv) * a.BS;
          else record_error(a.status, KVC_ERR_BOUNDS);
        }
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, slot >= 0);
        if (lane == 0) valid_s[st] = ok;
        constexpr int RPI = 32 / CH;
        const int col = lane % CH;
#pragma unroll 2
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
    look(t0);
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
      for (int o = 1; o < CH; o <<= 1) top = max(top, __shfl_xor_sync(__activemask(), top, o));
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
    // two products' operands of eight rows' queries (products ks and ks + 1)
    auto query8 = [&](int nr, int ks, uint32_t (&f)[4]) {
      ldsm4(qhbase + swz<D>(8 * nr + (lane & 7), 2 * ks + (lane >> 3)), f);
    };
    auto query16 = [&](int nr, int ks, uint32_t &b0, uint32_t &b1) {  // one product's, bf16
      const int row = 8 * nr + g8, x = rt * a.rstep + row;
      const uint16_t *p = a.q + ((int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G) * D + 16 * ks + 2 * quad;
      b0 = row < n_rows ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
      b1 = row < n_rows ? __ldg(reinterpret_cast<const uint32_t *>(p + 8)) : 0u;
    };
    uint32_t qf[NR == 1 ? KS / 2 : 1][4];  // eight rows keep q in registers
    if (NR == 1)
#pragma unroll
      for (int i = 0; i < KS / 2; i++) query8(0, 2 * i, qf[NR == 1 ? i : 0]);
    bool hist = t0 < th;  // O's columns lie as the history's products leave them

    // This thread's rows 8·nr + 2·quad + {0, 1}: the softmax's reference, its part of the sum,
    // how far O's reference lies above the softmax's; O of its columns.  References are the
    // warp's own.
    float o[CH8][NR][4], ref[NR][2], l[NR][2], off[NR][2], rs[NR][2];
    bool rounded = false;  // (warp-uniform) some reference is so large that differences need care
    bool infinite = false;  // (warp-uniform) values of nodes were left out that are not finite
#pragma unroll
    for (int nr = 0; nr < NR; nr++) {
#pragma unroll
      for (int e = 0; e < 2; e++) {
        ref[nr][e] = kQ8Unset;
        l[nr][e] = off[nr][e] = 0.f;
        rs[nr][e] = row_s[8 * nr + 2 * quad + e];
      }
#pragma unroll
      for (int n = 0; n < CH8; n++) o[n][nr][0] = o[n][nr][1] = o[n][nr][2] = o[n][nr][3] = 0.f;
    }
    // From the columns of the history's products (16n + 2·g8 and the next one, in elements
    // 0, 1 and 2, 3) to the usual ones (16n + g8 and 16n + 8 + g8).
    auto usual = [&]() {
      const int from = ((lane >> 3) << 2) | quad;
#pragma unroll
      for (int n = 0; n < CH8; n++)
#pragma unroll
        for (int nr = 0; nr < NR; nr++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const float v0 = o[n][nr][e], v1 = o[n][nr][2 + e];
            const float x0 = __shfl_sync(0xFFFFFFFFu, v0, from), x1 = __shfl_sync(0xFFFFFFFFu, v1, from);
            const float y0 = __shfl_sync(0xFFFFFFFFu, v0, from + 16), y1 = __shfl_sync(0xFFFFFFFFu, v1, from + 16);
            o[n][nr][e] = g8 & 1 ? x1 : x0;
            o[n][nr][2 + e] = g8 & 1 ? y1 : y0;
          }
      hist = false;
    };
    // Logits s become weights in place.  The factor of a logit is kz[key]·rs[row] (one of
    // them 1), that of V sv[key]; keys 8i + g8 of the tile, NK eights.
    auto softmax = [&](auto Nk, auto &s, const auto &kz, const auto &sv, bool scaled, bool masked,
                       const auto &vis) {
      constexpr int NK = decltype(Nk)::value;
      auto weights = [&](bool raised, float (&sum)[NR][2], float (&w)[NK / 2][NR][4]) {
        bool fine = true;
#pragma unroll
        for (int nr = 0; nr < NR; nr++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const float f = ex2(-0.5f * off[nr][e]);
            float most = 0.f;
            sum[nr][e] = 0.f;
#pragma unroll
            for (int i = 0; i < NK; i++) {
              float &x = s[i / 2][nr][2 * (i & 1) + e];
              const float k = scaled ? kz[i] * rs[nr][e] : a.zscale;
              float z = raised ? __fsub_rn(__fmul_rn(x, k), ref[nr][e]) : fmaf(x, k, -ref[nr][e]);
              if (masked && !((vis[nr][e] >> (8 * i + g8)) & 1u)) z = -INFINITY;
              z = ex2(z);
              sum[nr][e] += z;
              // (in halves: the scale times the whole factor may pass fp32; times a half, only
              // where the weight is 0, and 0·inf is 0.  A NaN is in the sum.)
              z = scaled ? fmaxf((z * f) * (sv[i] * f), 0.f) : z * f * f;
              most = fmaxf(most, z);
              w[i / 2][nr][2 * (i & 1) + e] = z;
            }
            fine = fine && sum[nr][e] <= kQ8Most && most <= kQ8Most;
          }
        return __all_sync(0xFFFFFFFFu, fine);
      };
      float sum[NR][2], w[NK / 2][NR][4];
      // (a row that has seen nothing makes an infinite weight of the first key it sees)
      if (rounded || !weights(false, sum, w)) {
        bool large = false;
#pragma unroll
        for (int nr = 0; nr < NR; nr++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float z[NK], mx = -INFINITY, mv = -INFINITY;
#pragma unroll
            for (int i = 0; i < NK; i++) {
              z[i] = __fmul_rn(s[i / 2][nr][2 * (i & 1) + e], scaled ? kz[i] * rs[nr][e] : a.zscale);
              if (masked && !((vis[nr][e] >> (8 * i + g8)) & 1u)) z[i] = -INFINITY;
              mx = fmaxf(mx, z[i]);
            }
#pragma unroll
            for (int o2 = 4; o2 < 32; o2 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o2));
            // (a large reference is the largest rounded product itself: its difference is 0)
            const float now = fmaxf(ref[nr][e], fabsf(mx) < kQ8Round ? mx - kQ8Room : mx);
#pragma unroll
            for (int i = 0; i < NK; i++)
              if (z[i] > -INFINITY) mv = fmaxf(mv, __fsub_rn(z[i], now) + (scaled ? lg2(sv[i]) : 0.f));
#pragma unroll
            for (int o2 = 4; o2 < 32; o2 <<= 1) mv = fmaxf(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, o2));
            const float d = ref[nr][e] - now;
            const float up = fminf(fmaxf(fmaxf(mv - kQ8Room, d + off[nr][e]), -125.f), 125.f);
            const float f = ex2(d + off[nr][e] - up);
            l[nr][e] *= ex2(d);
#pragma unroll
            for (int n = 0; n < CH8; n++) {
              o[n][nr][e] *= f;
              o[n][nr][2 + e] *= f;
            }
            ref[nr][e] = now;
            off[nr][e] = up;
            large = large || (now != kQ8Unset && !(fabsf(now) < kQ8Round));
          }
        rounded = __any_sync(0xFFFFFFFFu, large);
        weights(true, sum, w);
      }
#pragma unroll
      for (int nr = 0; nr < NR; nr++)
#pragma unroll
        for (int e = 0; e < 2; e++) l[nr][e] += sum[nr][e];
#pragma unroll
      for (int i = 0; i < NK / 2; i++)
#pragma unroll
        for (int nr = 0; nr < NR; nr++)
#pragma unroll
          for (int e = 0; e < 4; e++) s[i][nr][e] = w[i][nr][e];
    };

    int st = 0;
    for (int t = t0; t < t1; t++) {
      cp_wait<kQ8Stages - 2>();
      if ((boxed >> st) & 1u) {
        if (!mbar_wait_bounded(full + 8 * st, (phase >> st) & 1u, failed)) {
          *failed = 1;
          record_error(a.status, KVC_ERR_TIMEOUT);
        }
        phase ^= 1u << st;
      }
      __syncwarp();  // the stage has landed, and every lane is done with the one before it
      const int nx = t + kQ8Stages - 1;
      if (nx < t1) issue(nx, (st + kQ8Stages - 1) % kQ8Stages);
      cp_commit();
      const uint32_t okb = valid_s[st];
      const uint32_t kb = ring + st * kQ8Stage;
      if (t < th) {
        const uint32_t vb = kb + kQ8Keys * D;
        constexpr int MK = kQ8Keys / 16;  // sixteens of positions
        float s[MK][NR][4];
#pragma unroll
        for (int i = 0; i < MK; i++)
#pragma unroll
          for (int nr = 0; nr < NR; nr++) s[i][nr][0] = s[i][nr][1] = s[i][nr][2] = s[i][nr][3] = 0.f;
#pragma unroll
        for (int hi = 0; hi < KS / 4; hi++) {  // four products from a 16-byte piece of each row
          uint32_t kw[2 * MK][4];
#pragma unroll
          for (int i = 0; i < 2 * MK; i++) lds128(kb + swz8<D>(8 * i + g8, 4 * hi + quad), kw[i]);
#pragma unroll
          for (int k2 = 0; k2 < 2; k2++) {
            uint32_t qb[NR][4];
#pragma unroll
            for (int nr = 0; nr < NR; nr++) {
              if (NR == 1) {
#pragma unroll
                for (int e = 0; e < 4; e++) qb[nr][e] = qf[NR == 1 ? 2 * hi + k2 : 0][e];
              } else {
                query8(nr, 4 * hi + 2 * k2, qb[nr]);
              }
            }
#pragma unroll
            for (int k1 = 0; k1 < 2; k1++) {
              const int ks = 2 * k2 + k1;
#pragma unroll
              for (int i = 0; i < MK; i++) {
                const uint32_t ka[4] = {e4m3x2_f16x2(kw[2 * i][ks]), e4m3x2_f16x2(kw[2 * i + 1][ks]),
                                        e4m3x2_f16x2_hi(kw[2 * i][ks]), e4m3x2_f16x2_hi(kw[2 * i + 1][ks])};
#pragma unroll
                for (int nr = 0; nr < NR; nr++) mma16816h(s[i][nr], ka, qb[nr][2 * k1], qb[nr][2 * k1 + 1]);
              }
            }
          }
        }
        float kz[2 * MK], sv[2 * MK];  // scale·s_k·log2 e and s_v of this thread's positions
#pragma unroll
        for (int i = 0; i < 2 * MK; i++) {
          const float2 f = scale_s[st * kQ8Keys + 8 * i + g8];
          kz[i] = f.x * a.zscale;
          sv[i] = f.y;
        }
        uint32_t vis[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; nr++) vis[nr][0] = vis[nr][1] = okb;
        if (okb == 0xFFFFFFFFu) softmax(std::integral_constant<int, 2 * MK>(), s, kz, sv, true, false, vis);
        else softmax(std::integral_constant<int, 2 * MK>(), s, kz, sv, true, true, vis);
#pragma unroll
        for (int i = 0; i < MK; i++) {
          uint32_t pb[NR][2];
#pragma unroll
          for (int nr = 0; nr < NR; nr++) {
            pb[nr][0] = transpose8(pack_f16x2(s[i][nr][0], s[i][nr][1]));
            pb[nr][1] = transpose8(pack_f16x2(s[i][nr][2], s[i][nr][3]));
          }
#pragma unroll
          for (int n = 0; n < CH8; n += 2) {
            // two positions by two neighbouring columns a register; after the exchange of the
            // middle bytes its halves are the operands of the even and of the odd columns
            uint32_t b[4];
            ldsm4t(vb + swz8<D>(i * 16 + (lane & 15), n + (lane >> 4)), b);
#pragma unroll
            for (int u = 0; u < 4; u++) b[u] = __byte_perm(b[u], 0, 0x3120);
#pragma unroll
            for (int u = 0; u < 2; u++) {
              const uint32_t va[4] = {e4m3x2_f16x2(b[2 * u]), e4m3x2_f16x2_hi(b[2 * u]),
                                      e4m3x2_f16x2(b[2 * u + 1]), e4m3x2_f16x2_hi(b[2 * u + 1])};
#pragma unroll
              for (int nr = 0; nr < NR; nr++) mma16816h(o[n + u][nr], va, pb[nr][0], pb[nr][1]);
            }
          }
        }
      } else {
        if (hist) usual();
        const uint32_t vb = kb + KT * D * 2;
        const int p0 = (t - th) * a.tile + warp * KT;
        constexpr int MK = KT / 16;
        float s[MK][NR][4];
#pragma unroll
        for (int i = 0; i < MK; i++)
#pragma unroll
          for (int nr = 0; nr < NR; nr++) s[i][nr][0] = s[i][nr][1] = s[i][nr][2] = s[i][nr][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          uint32_t qb[NR][2];
#pragma unroll
          for (int nr = 0; nr < NR; nr++) query16(nr, ks, qb[nr][0], qb[nr][1]);
#pragma unroll
          for (int i = 0; i < MK; i++) {
            uint32_t ka[4];
            ldsm4(kb + swz<D>(i * 16 + (lane & 15), 2 * ks + (lane >> 4)), ka);
#pragma unroll
            for (int nr = 0; nr < NR; nr++) mma16816(s[i][nr], ka, qb[nr][0], qb[nr][1]);
          }
        }
        uint32_t vis[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; nr++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int x = rt * a.rstep + 8 * nr + 2 * quad + e;
            vis[nr][e] = x < T * a.G ? visible_bits<KT>(a, x / a.G, q0, c, T, p0) & okb : 0u;
          }
        const float one[2 * MK] = {};  // (not read)
        softmax(std::integral_constant<int, 2 * MK>(), s, one, one, false, true, vis);
        // A node's V may hold infinities or NaN that some rows do not see, and a product 0·inf
        // would hand them to those rows.  A tile with such values takes the sum term by term,
        // over the rows' visible keys only, and leaves such a value to the run's end, where it is
        // added as it is, for a weight too small for fp32 is not 0.
        bool odd = false;
        if (p0 + KT > c) {
          for (int e = lane; e < KT * CH; e += 32) {
            uint32_t w[4];
            lds128(vb + swz<D>(e / CH, e % CH), w);
#pragma unroll
            for (int u = 0; u < 4; u++)
              odd |= (w[u] & 0x7F80u) == 0x7F80u || (w[u] & 0x7F800000u) == 0x7F800000u;
          }
          odd = __any_sync(0xFFFFFFFFu, odd);
        }
        if (odd) {
          infinite = true;
          auto add = [](float w, float v, float &acc) {
            acc = fabsf(v) < INFINITY ? fmaf(w, v, acc) : acc;
          };
#pragma unroll
          for (int nr = 0; nr < NR; nr++)
#pragma unroll
            for (int i = 0; i < 2 * MK; i++)
#pragma unroll 1
              for (int k = 0; k < 8; k++) {  // key 8i + k, its weights in the lanes 4k + quad
                const float w0 = __shfl_sync(0xFFFFFFFFu, s[i / 2][nr][2 * (i & 1)], 4 * k + quad);
                const float w1 = __shfl_sync(0xFFFFFFFFu, s[i / 2][nr][2 * (i & 1) + 1], 4 * k + quad);
                const bool s0 = (vis[nr][0] >> (8 * i + k)) & 1u, s1 = (vis[nr][1] >> (8 * i + k)) & 1u;
#pragma unroll
                for (int n = 0; n < CH8; n++)
#pragma unroll
                  for (int hf = 0; hf < 2; hf++) {
                    uint16_t v;
                    asm volatile("ld.shared.u16 %0, [%1];"
                                 : "=h"(v)
                                 : "r"(vb + swz<D>(8 * i + k, 2 * n + hf) + 2 * g8));
                    const float vf = bf16_lo(v);
                    if (s0) add(w0, vf, o[n][nr][2 * hf]);
                    if (s1) add(w1, vf, o[n][nr][2 * hf + 1]);
                  }
              }
        } else {
#pragma unroll
          for (int i = 0; i < MK; i++) {
            uint32_t pb[NR][2];
#pragma unroll
            for (int nr = 0; nr < NR; nr++) {
              pb[nr][0] = transpose8(pack_bf16x2(s[i][nr][0], s[i][nr][1]));
              pb[nr][1] = transpose8(pack_bf16x2(s[i][nr][2], s[i][nr][3]));
            }
#pragma unroll
            for (int n = 0; n < CH8; n++) {
              uint32_t va[4];
              ldsm4t(vb + swz<D>(i * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * n + ((lane >> 3) & 1)), va);
#pragma unroll
              for (int nr = 0; nr < NR; nr++) mma16816(o[n][nr], va, pb[nr][0], pb[nr][1]);
            }
          }
        }
      }
      st = (st + 1) % kQ8Stages;
    }
    cp_wait<0>();
    if (hist) usual();
    __syncthreads();  // every warp is done with the ring: it takes the warps' O

    float *o_s = reinterpret_cast<float *>(sm) + warp * R * D;
#pragma unroll
    for (int nr = 0; nr < NR; nr++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float sum = l[nr][e];
#pragma unroll
        for (int o2 = 4; o2 < 32; o2 <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o2);
        // O, on its own reference so far, becomes the mean of the warp's values: sums on the
        // softmax's reference would pass fp32 where |v| passes 2^113
        const float inv = sum == 0.f ? 0.f : 1.f / sum, f = ex2(off[nr][e]);
        const int row = 8 * nr + 2 * quad + e;
        if (g8 == 0) ml_s[warp * R + row] = make_float2(ref[nr][e] == kQ8Unset ? -INFINITY : ref[nr][e], sum);
#pragma unroll
        for (int n = 0; n < CH8; n++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++)
            o_s[row * D + ((16 * n + 8 * hf + g8) ^ (quad << 3))] = o[n][nr][2 * hf + e] * inv * f;
      }
    if (infinite) add_infinite<D, KT>(a, o_s, bt, t0, t1, th, h, rt, n_rows, q0, c, T);
    __syncthreads();
    const bool whole = !CL && t0 == 0 && t1 == n_kt;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (g != run0);
    for (int e = tid; e < n_rows * (D / 4); e += kQ8Threads) {
      const int row = e / (D / 4), d4 = (e % (D / 4)) * 4;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kQ8Warps; w++) mx = fmaxf(mx, ml_s[w * R + row].x);
      const float base = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f, share[kQ8Warps];
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kQ8Warps; w++) {
        const float2 ml = ml_s[w * R + row];
        share[w] = ml.y == 0.f ? 0.f : ml.y * ex2(ml.x - base);
        sum += share[w];
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      auto part = [&](int w) {
        return *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sm) + (w * R + row) * D +
                                                 (d4 ^ (((row >> 1) & 3) << 3)));
      };
#pragma unroll
      for (int w = 0; w < kQ8Warps; w++) {
        const float2 ml = ml_s[w * R + row];
        // (this warp saw nothing of the row; logits that are all NaN leave a NaN sum)
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        add_part(acc, part(w), share[w] * inv);
      }
      if (any_nan(acc)) {  // perhaps an infinity of no weight
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kQ8Warps; w++) {
          const float2 ml = ml_s[w * R + row];
          if (ml.x == -INFINITY && ml.y == 0.f) continue;
          add_part_inf(acc, part(w), share[w] * inv);
        }
      }
      if (whole) {
        const int x = rt * a.rstep + row;
        const int64_t qr = (int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G;
        *reinterpret_cast<uint2 *>(a.out + qr * D + d4) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        if (d4 == 0) a.lse[qr] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
      } else if (CL) {
        *reinterpret_cast<float4 *>(sm + S::kClO + (row * D + d4) * 4) = acc;
        if (d4 == 0) reinterpret_cast<float2 *>(sm + S::kClMl)[row] = make_float2(mx, sum);
      } else {
        *reinterpret_cast<float4 *>(a.part_o + (slot * R + row) * D + d4) = acc;
        if (d4 == 0) a.part_ml[slot * R + row] = make_float2(mx, sum);
      }
    }
    if constexpr (CL) {
      // the cluster's CTAs hold the unit's parts: added up in order, the elements dealt out to
      // all of them
      __syncwarp();
      cluster_sync_all();
      const int n_cl = (int)cluster_nrank();
      const uint32_t o_at = smem_u32(sm + S::kClO), ml_at = smem_u32(sm + S::kClMl);
      for (int e = (int)cluster_rank() * kQ8Threads + tid; e < n_rows * (D / 4); e += n_cl * kQ8Threads) {
        const int row = e / (D / 4), d4 = (e % (D / 4)) * 4;
        float mx = -INFINITY;
        float2 mls[16];  // (asked for at once)
        float4 vs[16];
#pragma unroll
        for (int k = 0; k < 16; k++)
          if (k < n_cl) {
            mls[k] = ld_cluster_f2(mapa_u32(ml_at + row * 8, k));
            vs[k] = ld_cluster_f4(mapa_u32(o_at + (row * D + d4) * 4, k));
            mx = fmaxf(mx, mls[k].x);
          }
        const float base = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; k++) {
          if (k >= n_cl) break;
          mls[k].y *= ex2(mls[k].x - base);
          sum += mls[k].y;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int k = 0; k < 16; k++) {
          if (k >= n_cl) break;
          add_part(acc, vs[k], mls[k].y * inv);
        }
        if (any_nan(acc)) {
          acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 16; k++) {
            if (k >= n_cl) break;
            add_part_inf(acc, vs[k], mls[k].y * inv);
          }
        }
        const int x = rt * a.rstep + row;
        const int64_t qr = (int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G;
        *reinterpret_cast<uint2 *>(a.out + qr * D + d4) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        if (d4 == 0) a.lse[qr] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
      }
      __syncwarp();
      cluster_sync_all();  // (no CTA leaves while another reads its part)
      break;
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
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (O's place is the ring again)
      __syncthreads();
    }
  }
  if (*failed)  // this warp's copies finish before its memory is released
    for (int i = 0; i < kQ8Stages; i++) {
      mbar_drain(full + 8 * i, 0);
      mbar_drain(full + 8 * i, 1);
    }
}

// Rows per tile and grid of a call.
void q8_plan(int n_req, int max_blocks8, int max_blocks, int max_tree, int H, int Hq, int D, int BS,
             int &rows, int &tile, int &n_cta, int &max_rt) {
  const int64_t R = (int64_t)max_tree * (Hq / H);
  rows = (int)std::min<int64_t>((R + 7) / 8 * 8, 32);
  tile = kQ8Warps * (2048 / D);
  max_rt = (int)((R + rows - 1) / rows);
  const int64_t kt = ((int64_t)max_blocks8 * BS + kQ8Warps * kQ8Keys - 1) / (kQ8Warps * kQ8Keys) +
                     ((int64_t)max_blocks * BS + tile - 1) / tile;
  n_cta = (int)std::min<int64_t>(q8_ctas(rows / 8) * device_sm_count(), (int64_t)n_req * H * max_rt * kt);
}

// Boxes of `box` rows of a head's block, D bytes, swizzled as swz8 says.
bool rows8_map(CUtensorMap *m, const void *pool, int64_t rows, int D, int box) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)D};
  cuuint32_t bx[2] = {(cuuint32_t)D, (cuuint32_t)box}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(pool), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of the cluster that shares a unit, 0: the tiles are dealt out and joined by a second
// launch.  In the time of a tile that a CTA works on alone (1.05 us; `beat` tiles are what the
// memory takes to give one to every CTA that the GPU holds).  Dealt out: an even share, 10 for
// the two launches, 4.5 for every unit that a CTA meets.  Clusters: waves of CTAs, each its
// share of a unit's tiles, 6 to begin and end where it waits for itself, 4 where for memory.
// One token, 8 KV and 32 query heads, D 128, in us dealt out and by 1, 2, 4, 8 and 16: one
// request of 200 10, 9, 9, 7, 7, 8; of 4096 12, 43, 25, 16, 12, 11; 4 of 8192 23, 77, 43,
// 25, 19, 28; 16 of 4096 36, 44, 32, 45, 46, 77; 57 of 1024 (a CTA each) 29, 26, 34, 55, 88,
// 183; 64 of 1024 38, 44, 46, 59, 100, 206; 128 of 200 40, 30, 49, 78, 151, 382.  The tiles are
// the tables' width, for the lengths lie on the device; these figures are of tables as long as
// the requests.
int q8_cluster(const Q8Args &a, int max_rt, int D) {
  if (max_rt > 1 || a.rows > 16) return 0;  // (a cluster takes one row tile; more rows leave it to the even deal)
  const double units = (double)a.n_req * a.H, all = q8_ctas(a.rows / 8) * (double)device_sm_count();
  const double kt = ceil((double)a.max_blocks8 * a.BS / (kQ8Warps * kQ8Keys)) +
                    ceil((double)a.max_blocks * a.BS / a.tile);
  const double beat = 2.33 * D / 128, even = units * kt / all;
  int best = 0;
  double least = std::max(even * beat, ceil(even)) + 10 + 4.5 * units / all;
  for (int S = 1; S <= 16 && S < 2 * kt; S *= 2) {
    // (a GPC's 16 to 20 SMs hold fewer large clusters)
    const double room = all * (S == 16 ? 0.42 : S == 8 ? 0.84 : S == 4 ? 0.95 : 1);
    const double share = ceil(kt / S), waves = units * S / room, rest = waves - floor(waves);
    auto wave = [&](double full) { return std::max(share + 6, full * room / all * beat * share + 4); };
    const double cost = floor(waves) * wave(1) + (rest > 0 ? wave(rest) : 0) + (S == 16 ? 1.5 : 0);
    if (cost < least) {
      least = cost;
      best = S;
    }
  }
  return units * best <= INT32_MAX ? best : 0;
}

template <int D, int NR, bool CL>
cudaError_t launch_q8_rows(const Q8Args &a, const CUtensorMap &tm_k, const CUtensorMap &tm_v, int cluster,
                           cudaStream_t s) {
  constexpr int smem = Q8Smem<D, NR>::kBytes;
  auto *kern = k_q8_rows<D, NR, CL>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && cluster > 8)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL ? (unsigned)(a.n_req * a.H * cluster) : (unsigned)a.n_cta);
  cfg.blockDim = dim3(kQ8Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, a);
}
template <int D>
cudaError_t launch_q8(const Q8Args &a, int cluster, cudaStream_t s) {
  CUtensorMap tm_k{}, tm_v{};
  const int64_t rows = a.n_blocks8 * a.H * a.BS;
  if (a.box8 && !(rows8_map(&tm_k, a.k8, rows, D, a.box8) && rows8_map(&tm_v, a.v8, rows, D, a.box8)))
    return cudaErrorUnknown;
  switch (a.rows / 8) {
    case 1: return cluster ? launch_q8_rows<D, 1, true>(a, tm_k, tm_v, cluster, s)
                           : launch_q8_rows<D, 1, false>(a, tm_k, tm_v, 0, s);
    case 2: return cluster ? launch_q8_rows<D, 2, true>(a, tm_k, tm_v, cluster, s)
                           : launch_q8_rows<D, 2, false>(a, tm_k, tm_v, 0, s);
    case 3: return launch_q8_rows<D, 3, false>(a, tm_k, tm_v, 0, s);
    default: return launch_q8_rows<D, 4, false>(a, tm_k, tm_v, 0, s);
  }
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
  // (a box's rows lie in one block, and a row's number fits the box's coordinate)
  // (64 requests of 4096: pages of 32 and 16 95 us, of 8 98, of 12 and 4 by cp.async 99 and 100)
  a.box8 = n_blocks8 * H * BS > INT32_MAX ? 0 : BS % 32 == 0 ? 32 : BS % 16 == 0 ? 16 : BS % 8 == 0 ? 8 : 0;
  const int cluster = q8_cluster(a, max_rt, D);
  const cudaError_t e = D == 128 ? launch_q8<128>(a, cluster, s) : launch_q8<64>(a, cluster, s);
  if (e != cudaSuccess || cluster) return e;
  return launch_join(a, D, max_rt, s);
}

}  // namespace kvc
