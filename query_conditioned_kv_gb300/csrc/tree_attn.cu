// tree_attn.cu — attention of drafted token trees over a paged KV cache, one
// layer.  Row i of request r sees the c cached positions and the nodes its
// mask marks:
//   z_p = scale·q·k_p,  lse = ln Σ_p exp z_p,  out = Σ_p exp(z_p − lse)·v_p
//
// The T·G rows (node, head of the group) that share a KV head share every key
// and value row, so the unit of work is (request, KV head, row tile) and K
// and V are read once per unit.  With few rows the bound is the K and V
// stream: 4·D bytes per key against 4·D·rows operations.
//
// Split.  A unit's positions are cut into tiles of 64 (D 128) or 128 (D 64)
// keys; all tiles of all units, in order, are dealt out in equal contiguous
// runs to the CTAs, whatever the lengths of the requests: a single long
// request uses the whole GPU and a ragged batch ends together.  A run that
// holds all of a unit writes its result; otherwise it writes a partial
// (max, sum, unnormalised O in fp32) to the workspace, at most two per CTA,
// and k_tree_join adds a unit's partials in order.  No atomics: the result
// does not depend on timing.
//
// k_tree_rows (up to 32 rows a tile): each of a CTA's four warps streams its
// own quarter of every tile through a private cp.async ring (3 stages of
// 8 KB, so about 128 KB in flight per SM with two CTAs) and keeps its own
// softmax statistics and accumulators; no barrier until the run ends.  The
// products are mma.sync m16n8k16 with fp32 accumulators: at 16 rows the
// tensor work per key is a few per cent of the time its bytes take, so the
// narrow instruction, which needs no shared-memory round trip for the
// weights, is enough.
#include <math.h>

#include <algorithm>

#include "kvc_internal.cuh"
#include "mma_ptx.cuh"
#include "tc_ptx.cuh"

namespace kvc {
namespace {

using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
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
  float zscale;  // scale·log2(e)
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

__device__ __forceinline__ int64_t run_start(int64_t total, int n_cta, int cta) {
  return total * cta / n_cta;
}
// The CTA whose run holds tile t.
__device__ __forceinline__ int run_owner(int64_t total, int n_cta, int64_t t) {
  int c = (int)(t * n_cta / total);
  while (c + 1 < n_cta && run_start(total, n_cta, c + 1) <= t) c++;
  while (c > 0 && run_start(total, n_cta, c) > t) c--;
  return c;
}

// Tiles of request r, all heads.
__device__ __forceinline__ int64_t request_tiles(const TreeArgs &a, int r) {
  int n_rt, n_kt;
  tree_tiles(a, r, n_rt, n_kt);
  return (int64_t)a.H * n_rt * n_kt;
}

constexpr int kRowWarps = 4;
constexpr int kRowThreads = kRowWarps * 32;
constexpr int kRowStages = 3;
constexpr int kWarpStage = 8192;  // bytes of one warp's stage: K rows, then V rows

template <int D, int MT>
struct RowSmem {
  static constexpr int kRing = kRowWarps * kRowStages * kWarpStage;
  static constexpr int kQ = kRing;                       // MT·16 rows of q
  static constexpr int kMisc = kQ + MT * 16 * D * 2;     // scan scratch [66] int64
  static constexpr int kValid = kMisc + 66 * 8;          // valid keys per (warp, stage)
  static constexpr int kMl = kValid + kRowWarps * kRowStages * 4;  // (max, sum) per (warp, row)
  static constexpr int kBytes = kMl + kRowWarps * MT * 16 * 8;
  static_assert(kRowWarps * MT * 16 * D * 4 <= kRing, "the warps' O fits the ring");
};

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

template <int D, int MT>
__global__ void __launch_bounds__(kRowThreads, 2)
k_tree_rows(TreeArgs a) {
  using S = RowSmem<D, MT>;
  constexpr int KT = 2048 / D, KS = D / 16, NT = D / 8, CH = D / 8;
  constexpr int R = MT * 16;
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t *sh = reinterpret_cast<int64_t *>(sm + S::kMisc);
  const uint32_t ring = smem_u32(sm) + warp * kRowStages * kWarpStage;
  uint32_t *valid_s = reinterpret_cast<uint32_t *>(sm + S::kValid) + warp * kRowStages;
  const uint32_t qbase = smem_u32(sm + S::kQ);
  float2 *ml_s = reinterpret_cast<float2 *>(sm + S::kMl);

  asm volatile("griddepcontrol.launch_dependents;");
  if (blockIdx.x == 0)  // one report per bad request
    for (int r = tid; r < a.n_req; r += kRowThreads) {
      int c, q0, T;
      if (!tree_request(a, r, c, q0, T)) record_error(a.status, KVC_ERR_BOUNDS);
    }
  int64_t total = 0, before;
  for (int x = tid; x < a.n_req; x += kRowThreads) total += request_tiles(a, x);
  total = block_sum(total, sh);
  const int n_cta = (int)min((int64_t)a.n_cta, total);  // every run holds a tile
  if ((int)blockIdx.x >= n_cta) return;
  const int64_t run0 = run_start(total, n_cta, blockIdx.x);
  const int64_t run1 = run_start(total, n_cta, blockIdx.x + 1);
  int r;
  block_find(a.n_req, run0, sh, [&](int x) { return request_tiles(a, x); }, r, before);

  const int64_t n_blocks = a.n_slots / a.BS;
  int64_t g = run0;  // next tile of the run
  int c, q0, T, n_rt, n_kt;
  tree_request(a, r, c, q0, T);
  tree_tiles(a, r, n_rt, n_kt);
  int unit = (int)((g - before) / n_kt);  // h·n_rt + row tile
  int t0 = (int)((g - before) % n_kt);
  while (g < run1) {
    const int h = unit / n_rt, rt = unit % n_rt;
    const int t1 = (int)min((int64_t)n_kt, t0 + (run1 - g));
    const int n_rows = min(a.rstep, T * a.G - rt * a.rstep);
    const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
    const int end = c + T;

    // issue one stage: this warp's KT keys of tile t
    auto issue = [&](int t, int st) {
      const int p0 = t * a.tile + warp * KT;
      int32_t slot = -1;
      if (lane < KT && p0 + lane < end) {
        const int p = p0 + lane;
        const int32_t b = bt[p / a.BS];
        if (b >= 0 && b < n_blocks) slot = b * a.BS + p % a.BS;
        else record_error(a.status, KVC_ERR_BOUNDS);
      }
      const uint32_t ok = __ballot_sync(0xFFFFFFFFu, slot >= 0);
      if (lane == 0) valid_s[st] = ok;
      const uint32_t dst = ring + st * kWarpStage;
      constexpr int RPI = 32 / CH;  // rows one instruction of the warp copies
      const int col = lane % CH;
#pragma unroll
      for (int i = 0; i < KT / RPI; i++) {
        const int row = i * RPI + lane / CH;
        const int32_t sl = __shfl_sync(0xFFFFFFFFu, slot, row);
        const int64_t at = ((int64_t)max(sl, 0) * a.H + h) * D + col * 8;
        cp_async16(dst + swz<D>(row, col), a.kpool + at, sl >= 0);
        cp_async16(dst + KT * D * 2 + swz<D>(row, col), a.vpool + at, sl >= 0);
      }
    };
    const int n_t = t1 - t0;
#pragma unroll
    for (int s = 0; s < kRowStages - 1; s++) {
      if (s < n_t) issue(t0 + s, s);
      cp_commit();
    }
    // the row tile's queries
    for (int e = tid; e < R * CH; e += kRowThreads) {
      const int row = e / CH, col = e % CH, x = rt * a.rstep + row;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < n_rows)
        v = *reinterpret_cast<const uint4 *>(
            a.q + ((int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G) * D + col * 8);
      *reinterpret_cast<uint4 *>(sm + S::kQ + swz<D>(row, col)) = v;
    }
    __syncthreads();
    uint32_t qf[MT == 1 ? KS : 1][4];  // one row tile of 16 keeps q in registers
    if (MT == 1)
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
        ldsm4(qbase + swz<D>(lane % 16, 2 * ks + lane / 16), qf[MT == 1 ? ks : 0]);

    float o[MT][NT][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; n++) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    }

    int st = 0;
    for (int t = t0; t < t1; t++) {
      cp_wait<kRowStages - 2>();
      __syncwarp();  // the stage has landed, and every lane is done with the one before it
      const int nx = t + kRowStages - 1;
      if (nx < t1) issue(nx, (st + kRowStages - 1) % kRowStages);
      cp_commit();
      const uint32_t kb = ring + st * kWarpStage, vb = kb + KT * D * 2;
      const int p0 = t * a.tile + warp * KT;
      const uint32_t okb = valid_s[st];
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
            ldsm4(qbase + swz<D>(mt * 16 + lane % 16, 2 * ks + lane / 16), qa[mt]);
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
      // scale, mask, online softmax (rows lane/4 and lane/4 + 8 of each tile)
      const bool masked = p0 + KT > c || okb != (KT == 32 ? 0xFFFFFFFFu : (1u << (KT & 31)) - 1u);
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
#pragma unroll
        for (int n = 0; n < KT / 8; n++)
#pragma unroll
          for (int e = 0; e < 4; e++) s[mt][n][e] *= a.zscale;
        if (masked) {  // warp-uniform
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
            const int x = rt * a.rstep + mt * 16 + hf * 8 + lane / 4;
            uint32_t vis = 0;
            if (x < T * a.G) vis = visible_bits<KT>(a, x / a.G, q0, c, T, p0) & okb;
#pragma unroll
            for (int n = 0; n < KT / 8; n++)
#pragma unroll
              for (int e = 0; e < 2; e++)
                if (!((vis >> (n * 8 + 2 * (lane % 4) + e)) & 1u)) s[mt][n][hf * 2 + e] = -INFINITY;
          }
        }
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
          float mx = m[mt][hf];
#pragma unroll
          for (int n = 0; n < KT / 8; n++) mx = max3(mx, s[mt][n][hf * 2], s[mt][n][hf * 2 + 1]);
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
          const float base = mx == -INFINITY ? 0.f : mx;
          const float f = ex2(m[mt][hf] - base);
          m[mt][hf] = mx;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < KT / 8; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const float w = ex2(s[mt][n][hf * 2 + e] - base);
              s[mt][n][hf * 2 + e] = w;
              sum += w;
            }
          l[mt][hf] = l[mt][hf] * f + sum;
          if (!__all_sync(0xFFFFFFFFu, f == 1.f))
#pragma unroll
            for (int n = 0; n < NT; n++) {
              o[mt][n][hf * 2] *= f;
              o[mt][n][hf * 2 + 1] *= f;
            }
        }
      }
      // A node's V may hold infinities or NaN that some rows do not see, and a
      // product 0·inf would hand them to those rows.  A tile with such values
      // takes the sum term by term, over the rows' visible keys only.
      bool odd = false;
      if (p0 + KT > c) {
        for (int e = lane; e < KT * CH; e += 32) {
          const int row = e / CH;
          uint32_t w[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(vb + swz<D>(row, e % CH)));
#pragma unroll
          for (int u = 0; u < 4; u++)
            odd |= (w[u] & 0x7F80u) == 0x7F80u || (w[u] & 0x7F800000u) == 0x7F800000u;
        }
        odd = __any_sync(0xFFFFFFFFu, odd);
      }
      if (odd) {
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int kn = 0; kn < KT / 8; kn++)
            for (int kq = 0; kq < 4; kq++)
#pragma unroll
              for (int e = 0; e < 2; e++) {  // key 8·kn + 2·kq + e
                const int src = (lane & ~3) | kq;
                const float w0 = __shfl_sync(0xFFFFFFFFu, s[mt][kn][e], src);
                const float w1 = __shfl_sync(0xFFFFFFFFu, s[mt][kn][2 + e], src);
#pragma unroll
                for (int n = 0; n < NT; n++) {
                  uint32_t v;
                  asm volatile("ld.shared.u32 %0, [%1];"
                               : "=r"(v)
                               : "r"(vb + swz<D>(8 * kn + 2 * kq + e, n) + 4 * (lane % 4)));
                  if (w0 > 0.f) {
                    o[mt][n][0] = fmaf(w0, bf16_lo(v), o[mt][n][0]);
                    o[mt][n][1] = fmaf(w0, bf16_hi(v), o[mt][n][1]);
                  }
                  if (w1 > 0.f) {
                    o[mt][n][2] = fmaf(w1, bf16_lo(v), o[mt][n][2]);
                    o[mt][n][3] = fmaf(w1, bf16_hi(v), o[mt][n][3]);
                  }
                }
              }
      } else {
#pragma unroll
        for (int kk = 0; kk < KT / 16; kk++) {
          uint32_t pa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            pa[mt][0] = pack_bf16x2(s[mt][2 * kk][0], s[mt][2 * kk][1]);
            pa[mt][1] = pack_bf16x2(s[mt][2 * kk][2], s[mt][2 * kk][3]);
            pa[mt][2] = pack_bf16x2(s[mt][2 * kk + 1][0], s[mt][2 * kk + 1][1]);
            pa[mt][3] = pack_bf16x2(s[mt][2 * kk + 1][2], s[mt][2 * kk + 1][3]);
          }
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm4t(vb + swz<D>(kk * 16 + (lane & 15), n + (lane >> 4)), b);
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
              mma16816(o[mt][n], pa[mt], b[0], b[1]);
              mma16816(o[mt][n + 1], pa[mt], b[2], b[3]);
            }
          }
        }
      }
      st = (st + 1) % kRowStages;
    }
    cp_wait<0>();
    __syncthreads();  // every warp is done with the ring: it takes the warps' O

    float *o_s = reinterpret_cast<float *>(sm) + warp * R * D;
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        float sum = l[mt][hf];
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
        const int row = mt * 16 + hf * 8 + lane / 4;
        if (lane % 4 == 0) ml_s[warp * R + row] = make_float2(m[mt][hf], sum);
#pragma unroll
        for (int n = 0; n < NT; n++)
          *reinterpret_cast<float2 *>(o_s + row * D + ((n * 8 + 2 * (lane % 4)) ^ ((row & 3) << 3))) =
              make_float2(o[mt][n][hf * 2], o[mt][n][hf * 2 + 1]);
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == n_kt;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (g != run0);
    for (int e = tid; e < n_rows * (D / 4); e += kRowThreads) {
      const int row = e / (D / 4), d4 = (e % (D / 4)) * 4;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kRowWarps; w++) mx = fmaxf(mx, ml_s[w * R + row].x);
      const float base = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowWarps; w++) {
        const float2 ml = ml_s[w * R + row];
        if (ml.x == -INFINITY) continue;  // this warp saw nothing of the row
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
        const float inv = mx == -INFINITY ? 0.f : 1.f / sum;
        uint2 w2 = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2 *>(a.out + qr * D + d4) = w2;
        if (d4 == 0) a.lse[qr] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * kLn2;
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
        tree_request(a, r, c, q0, T);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- tcgen05
//
// k_tree_tc (more than 32 rows).  Per tile of 128 keys, both products with
// the rows as the N dimension:
//   Sᵀ[key][row] = K·Qᵀ          (M 128 keys,  N rows, K D)
//   Oᵀ[d][row] += Vᵀ·Pᵀ          (M D (64 twice), N rows, K 128 keys)
// so the tensor work grows with the rows instead of being padded to 128, and
// at 256 rows each instruction is the widest (N 256).  V and P are taken
// MN-major: V as it lies in the pool, P as the softmax threads hold it (one
// key per thread), written with 16-byte stores.
//
// A softmax thread owns one key (TMEM lane) and CW rows (columns), so a row's
// maximum is spread over 128 threads.  The exponent's reference is therefore
// not the running maximum but a fixed value per row, the maximum of the first
// tile, raised only when some logit exceeds it by 2^30: weights, their sums
// and O stay far inside fp32 and bf16 range (bf16 has fp32's exponents), and
// the result does not depend on the reference.  A per-tile vote of the
// warpgroup (one barrier) finds the tiles that must raise it; they take the
// exchange and rescale O in tensor memory.  The sums of the weights stay in
// registers per (key lane, row) and are reduced once per run.
//
// Warps: NW softmax warpgroups, two producer warps (cp.async, any page
// size), one MMA warp.  K and V tiles share one ring, in the order the MMA
// warp consumes them: K0 K1 V0 K2 V1 …

constexpr int kTtKeys = 128;
constexpr int kTtProd = 2;
constexpr int kTtThreads = 640;     // at most 4 softmax warpgroups, then the other warps
constexpr float kUnset = -1e30f;   // reference of a row that has seen nothing
constexpr float kExceed = 30.f;    // log2 of how far a logit may pass the reference

struct TreeTc {
  int NW;      // softmax warpgroups
  int NS;      // ring slots
  int PB, SB;  // P buffers, S buffers
  int box;     // rows of a TMA box (a divisor of the page size), 0: no TMA
  int q_nodes; // nodes of a row tile
  uint32_t idesc_s, idesc_o;  // without N
};

constexpr int kTtSlots = 8;  // ring slots, at most

// Head of the dynamic shared memory, at fixed offsets (few live registers);
// then the scratch of the warpgroups of 32 rows, P, the ring and q.
struct TreeTcHead {
  uint64_t full[kTtSlots], empty[kTtSlots], qfull, qempty;
  uint64_t sfull[2], sfree[2], pready[2], pvdone[2], ofree;
  int64_t scan[66];
  uint32_t tmem_holder;
  volatile int failed, odd, bad;
  float nb[256];  // −reference per row
};
constexpr uint32_t kTtHead = 2048;
static_assert(sizeof(TreeTcHead) <= kTtHead, "the head's room");

// Byte offsets (multiples of 1024) from the head.
struct TreeTcSmem {
  uint32_t p, ring, q, bytes;
  __host__ __device__ TreeTcSmem(int D, int rows, int NS, int PB) {
    p = kTtHead + (rows <= 128 ? 128 * 24 : 0);
    ring = p + PB * rows * (kTtKeys * 2);
    q = ring + NS * kTtKeys * D * 2;
    bytes = q + rows * D * 2;
  }
};

// MN-major operand with the 128-byte swizzle: 64 MN elements (128 B) by 8 K
// rows per 1024-byte atom; atoms along K are 1024 B apart, along MN `lbo`.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ bool named_sync_or(int id, int n, bool v) {
  return !named_sync_and(id, n, !v);
}

// Where a run stands: tiles [t0, t1) of one (request, KV head, row tile).
struct TreePos {
  int r, unit, n_rt, n_kt, c, q0, T;
  int64_t g, run0, run1;
  int t0;
  __device__ __forceinline__ void init(const TreeArgs &a, int64_t before) {
    tree_request(a, r, c, q0, T);
    tree_tiles(a, r, n_rt, n_kt);
    unit = (int)((g - before) / n_kt);
    t0 = (int)((g - before) % n_kt);
  }
  __device__ __forceinline__ int t1() const { return (int)min((int64_t)n_kt, t0 + (run1 - g)); }
  __device__ __forceinline__ int h() const { return unit / n_rt; }
  __device__ __forceinline__ int rt() const { return unit % n_rt; }
  __device__ __forceinline__ int rows(const TreeArgs &a) const {
    return min(a.rstep, T * a.G - rt() * a.rstep);
  }
  __device__ __forceinline__ void next(const TreeArgs &a) {
    const int e = t1();
    g += e - t0;
    t0 = 0;
    if (g < run1 && e == n_kt && ++unit == a.H * n_rt) {
      unit = 0;
      do {
        r++;
        tree_tiles(a, r, n_rt, n_kt);
      } while (n_rt == 0);
      tree_request(a, r, c, q0, T);
    }
  }
};

// 16 TMEM lanes × 8·NB columns (16x256b): register 4k + j of thread t holds
// lane t/4 + 8·(j ≥ 2), column 8k + 2·(t%4) + (j & 1).
template <int NB>
__device__ __forceinline__ void tmem_frag(uint32_t taddr, uint32_t (&r)[4 * NB]);
template <>
__device__ __forceinline__ void tmem_frag<4>(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <>
__device__ __forceinline__ void tmem_frag<8>(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                      uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

// x = z·zscale + nb of one 16-lane half (nb[2k + e]: rows 8k + 2·(t%4) + e),
// −inf where bit 4k + j of `see` is clear.  Scalar FMAs: the packed form
// costs more in register moves than it saves.
template <int NB>
__device__ __forceinline__ void tree_exponents(const uint32_t (&z)[4 * NB], float zs,
                                               const float (&nb)[2 * NB], bool masked, uint32_t see,
                                               float (&x)[4 * NB]) {
#pragma unroll
  for (int e = 0; e < 4 * NB; e++)
    x[e] = fmaf(__uint_as_float(z[e]), zs, nb[(e >> 2) * 2 + (e & 1)]);
  if (masked) {
    asm volatile("");  // a branch, not 4·NB selects in every tile
#pragma unroll
    for (int e = 0; e < 4 * NB; e++)
      if (!((see >> e) & 1u)) x[e] = -INFINITY;
  }
}

template <int D, int CW>
__global__ void __launch_bounds__(kTtThreads, 1)
k_tree_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
          const __grid_constant__ CUtensorMap tm_q, TreeArgs a, TreeTc p) {
  constexpr int CH = D / 8, KB = D / 64;
  constexpr uint32_t kSlot = kTtKeys * D * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TreeTcHead &sm = *reinterpret_cast<TreeTcHead *>(base);
  const TreeTcSmem at(D, a.rows, p.NS, p.PB);
  const uint32_t base_u = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nsw = p.NW * 4;  // softmax warps
  const uint32_t p_bytes = (uint32_t)a.rows * (kTtKeys * 2);

  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) {
    sm.failed = 0;
    sm.odd = 0;
    sm.bad = 0;
    for (int i = 0; i < p.NS; i++) {
      mbar_init(smem_u32(sm.full + i), kTtProd * 32);
      mbar_init(smem_u32(sm.empty + i), 1);
    }
    mbar_init(smem_u32(&sm.qfull), 1);
    mbar_init(smem_u32(&sm.qempty), 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(smem_u32(sm.sfull + i), 1);
      mbar_init(smem_u32(sm.sfree + i), nsw);
      mbar_init(smem_u32(sm.pready + i), nsw);
      mbar_init(smem_u32(sm.pvdone + i), 1);
    }
    mbar_init(smem_u32(&sm.ofree), nsw);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == nsw + kTtProd) alloc_tmem_cols(&sm.tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_holder;
  const uint32_t tmem_o = tmem + p.SB * a.rows;

  if (blockIdx.x == 0)  // one report per bad request
    for (int r = tid; r < a.n_req; r += blockDim.x) {
      int c, q0, T;
      if (!tree_request(a, r, c, q0, T)) record_error(a.status, KVC_ERR_BOUNDS);
    }
  int64_t total = 0;
  for (int x = tid; x < a.n_req; x += blockDim.x) total += request_tiles(a, x);
  total = block_sum(total, sm.scan);
  const int n_cta = (int)min((int64_t)a.n_cta, total);
  const bool works = (int)blockIdx.x < n_cta;
  TreePos pos{};
  if (works) {
    pos.run0 = pos.g = run_start(total, n_cta, blockIdx.x);
    pos.run1 = run_start(total, n_cta, blockIdx.x + 1);
    int64_t before;
    block_find(a.n_req, pos.g, sm.scan, [&](int x) { return request_tiles(a, x); }, pos.r, before);
    pos.init(a, before);
  }

bool ok = true;
  if (warp >= nsw && warp < nsw + kTtProd) {
    // ------------------------------------------------------- producers
    const int pw = warp - nsw;
    const int64_t n_blocks = a.n_slots / a.BS;
    constexpr int RPI = 32 / CH, NU = kTtKeys / (32 * kTtProd);  // this warp's blocks of 32 keys
    const int col = lane % CH;
    uint32_t rc = 0, qc = 0;
    uint32_t pend0 = 0, pend1 = 0;  // stages in flight, oldest first (the newest besides)
    auto hand = [&](uint32_t bar) {  // the stage's copies have landed: to the tensor core
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(bar);
    };
    auto flush = [&]() {
      if (pend1) {
        cp_wait<1>();
        hand(pend0);
        pend0 = pend1;
        pend1 = 0;
      }
      if (pend0) {
        cp_wait<0>();
        hand(pend0);
        pend0 = 0;
      }
    };
    // a full ring is waited for only after everything in flight is handed over
    auto acquire = [&](uint64_t *bar, uint32_t parity) {
      if (mbar_try(smem_u32(bar), parity)) return true;
      flush();
      return mbar_wait_bounded(smem_u32(bar), parity, &sm.failed);
    };
    auto committed = [&](uint64_t *bar) {
      cp_commit();
      if (pend1) {
        cp_wait<2>();
        hand(pend0);
        pend0 = pend1;
        pend1 = smem_u32(bar);
      } else if (pend0) {
        pend1 = smem_u32(bar);
      } else {
        pend0 = smem_u32(bar);
      }
    };
    while (pos.g < pos.run1 && ok) {
      const int t1 = pos.t1(), h = pos.h(), rt = pos.rt(), n_rows = pos.rows(a);
      const int32_t *bt = a.block_table + (int64_t)pos.r * a.max_blocks;
      const int end = pos.c + pos.T;
      int32_t blk[NU], ks[NU], vs[NU];  // block ids of the next tile; slots of this K, of this V
      auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < NU; u++) {
          const int pp = t * kTtKeys + pw * 32 + u * (32 * kTtProd) + lane;
          blk[u] = pp < end && t < t1 ? bt[pp / a.BS] : 0;
        }
      };
      auto resolve = [&](int t) {
#pragma unroll
        for (int u = 0; u < NU; u++) {
          const int pp = t * kTtKeys + pw * 32 + u * (32 * kTtProd) + lane;
          vs[u] = ks[u];
          ks[u] = -1;
          if (pp < end) {
            if (blk[u] >= 0 && blk[u] < n_blocks) {
              ks[u] = blk[u] * a.BS + pp % a.BS;
            } else {
              sm.bad = 1;  // (read by the softmax warps after this stage's product)
              record_error(a.status, KVC_ERR_BOUNDS);
            }
          }
        }
      };
      // One stage: TMA boxes of whole page rows where every key of the warp's
      // blocks is cached, else row by row with cp.async (zeros past the end).
      auto load = [&](const uint16_t *pool, const CUtensorMap *tm, int t, const int32_t (&slot)[NU]) {
        const int st = rc % p.NS;
        if (!(ok = acquire(sm.empty + st, ((rc / p.NS) & 1) ^ 1))) return;
        const uint32_t slot0 = (base_u + at.ring) + st * kSlot;
        bool whole = p.box > 0 && (t + 1) * kTtKeys <= pos.c;
        if (whole) {
#pragma unroll
          for (int u = 0; u < NU; u++) whole &= __all_sync(0xFFFFFFFFu, slot[u] >= 0);
        }
        if (whole) {
          const uint32_t bar = smem_u32(sm.full + st);
          if (lane == 0) mbar_expect_tx(bar, kSlot / kTtProd);
          else mbar_arrive(bar);
          __syncwarp();
          if (lane % p.box == 0)  // a box's first key
#pragma unroll
            for (int u = 0; u < NU; u++)
#pragma unroll
              for (int kb = 0; kb < KB; kb++)
                tma_load_3d(slot0 + kb * (kTtKeys * 128) +
                                (pw * 32 + u * (32 * kTtProd) + lane) * 128,
                            tm, kb * 64, h, slot[u], bar);
          __syncwarp();
          flush();  // (a stage copied row by row may still be in flight)
          rc++;
          return;
        }
        const uint32_t dst = slot0 + (col >> 3) * (kTtKeys * 128);
#pragma unroll
        for (int u = 0; u < NU; u++)
#pragma unroll
          for (int i = 0; i < 32 / RPI; i++) {
            const int row = i * RPI + lane / CH;
            const int32_t sl = __shfl_sync(0xFFFFFFFFu, slot[u], row);
            cp_async16(dst + (pw * 32 + u * (32 * kTtProd) + row) * 128 +
                           (((col & 7) ^ (row & 7)) << 4),
                       pool + ((int64_t)max(sl, 0) * a.H + h) * D + col * 8, sl >= 0);
          }
        committed(sm.full + st);
        rc++;
      };
      auto load_v = [&](int t, const int32_t (&slot)[NU]) {
        const uint32_t dst =
            (base_u + at.ring) + (rc % p.NS) * kSlot + (col >> 3) * (kTtKeys * 128);
        load(a.vpool, &tm_v, t, slot);
        if (!ok || (t + 1) * kTtKeys <= pos.c) return;
        // A node's V may hold infinities or NaN that some rows do not see: the
        // product gets zeros in their place, and the run's end adds them to
        // the rows that do.  Each thread looks at what it copied, before the
        // stage is handed over.
        cp_wait<0>();
        bool odd = false;
#pragma unroll 1
        for (int i = 0; i < NU * 32 / RPI; i++) {
          const int u0 = i * RPI + lane / CH;
          const int row = (u0 & 31) + pw * 32 + (u0 >> 5) * (kTtProd * 32);
          const uint32_t at = dst + row * 128 + (((col & 7) ^ (row & 7)) << 4);
          uint32_t w[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(at)
                       : "memory");
          bool mine = false;
#pragma unroll
          for (int u = 0; u < 4; u++) {
            if ((w[u] & 0x7F80u) == 0x7F80u) mine = true, w[u] &= 0xFFFF0000u;
            if ((w[u] & 0x7F800000u) == 0x7F800000u) mine = true, w[u] &= 0xFFFFu;
          }
          // (cached positions are seen by every row: their values stay)
          if (mine && t * kTtKeys + row >= pos.c) {
            odd = true;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
                         "r"(w[2]), "r"(w[3])
                         : "memory");
          }
        }
        if (odd) sm.odd = 1;
        flush();
      };
      // the row tile's queries, in one box of nodes × heads of the group; rows
      // past the request's own (another request's, or zeros) are columns that
      // the softmax leaves out
      auto load_q = [&]() {
        if (!(ok = acquire(&sm.qempty, (qc & 1) ^ 1))) return;
        if (pw == 0 && lane == 0) {
          const uint32_t bar = smem_u32(&sm.qfull);
          mbar_expect_tx(bar, p.q_nodes * a.G * D * 2);
#pragma unroll
          for (int kb = 0; kb < KB; kb++)
            tma_load_3d((base_u + at.q) + kb * (a.rows * 128), &tm_q, kb * 64, h * a.G,
                        pos.q0 + rt * p.q_nodes, bar);
        }
        qc++;
      };
      fetch(pos.t0);
      resolve(pos.t0);
      fetch(pos.t0 + 1);
      load(a.kpool, &tm_k, pos.t0, ks);
      if (ok) load_q();
      for (int t = pos.t0 + 1; t < t1 && ok; t++) {
        resolve(t);
        fetch(t + 1);
        load(a.kpool, &tm_k, t, ks);
        if (ok) load_v(t - 1, vs);
      }
      if (ok) load_v(t1 - 1, ks);
      pos.next(a);
    }
    flush();
    cp_wait<0>();
    if (!ok) sm.failed = 1;
  } else if (warp == nsw + kTtProd) {
    // ------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t rc = 0, qc = 0, sc = 0, vc = 0;  // ring slots, runs, S and PV products issued
      while (pos.g < pos.run1 && ok) {
        const int t0 = pos.t0, t1 = pos.t1(), n_rows = pos.rows(a);
        const uint32_t nbits = (uint32_t)((n_rows + 15) / 16 * 2) << 17;  // N / 8
        auto wait_slot = [&]() {
          const bool r = mbar_wait_bounded(smem_u32(sm.full + rc % p.NS), (rc / p.NS) & 1, &sm.failed);
          return r;
        };
        auto issue_s = [&](bool last) {
          const int b = sc % p.SB;
          if (!(ok = wait_slot())) return;
          if (!(ok = mbar_wait_bounded(smem_u32(sm.sfree + b), ((sc / p.SB) & 1) ^ 1, &sm.failed)))
            return;
          tc_fence_after();
          const uint32_t kb = (base_u + at.ring) + (rc % p.NS) * kSlot, qb = (base_u + at.q);
#pragma unroll
          for (int kk = 0; kk < 4 * KB; kk++)
            mma_bf16(tmem + b * a.rows,
                     smem_desc(kb + (kk >> 2) * (kTtKeys * 128) + (kk & 3) * 32),
                     smem_desc(qb + (kk >> 2) * (a.rows * 128) + (kk & 3) * 32), p.idesc_s | nbits,
                     kk > 0);
          mma_commit(smem_u32(sm.sfull + b));
          mma_commit(smem_u32(sm.empty + rc % p.NS));
          if (last) mma_commit(smem_u32(&sm.qempty));
          rc++;
          sc++;
        };
        auto issue_pv = [&](bool first) {
          if (!(ok = wait_slot())) return;
          if (first &&  // O's previous contents have been read
              !(ok = mbar_wait_bounded(smem_u32(&sm.ofree), (qc & 1) ^ 1, &sm.failed)))
            return;
          if (!(ok = mbar_wait_bounded(smem_u32(sm.pready + (vc & 1)), (vc >> 1) & 1, &sm.failed)))
            return;
          tc_fence_after();
          const uint32_t vb = (base_u + at.ring) + (rc % p.NS) * kSlot;
          const uint32_t pb = (base_u + at.p) + (vc % p.PB) * p_bytes;
#pragma unroll
          for (int kk = 0; kk < kTtKeys / 16; kk++)
            mma_bf16(tmem_o, smem_desc_mn(vb + kk * 2048, KB == 2 ? kTtKeys * 128 : 0),
                     smem_desc(pb + (kk >> 2) * (a.rows * 128) + (kk & 3) * 32), p.idesc_o | nbits,
                     !first || kk > 0);
          mma_commit(smem_u32(sm.pvdone + (vc & 1)));
          mma_commit(smem_u32(sm.empty + rc % p.NS));
          rc++;
          vc++;
        };
        ok = mbar_wait_bounded(smem_u32(&sm.qfull), qc & 1, &sm.failed);
        if (ok) issue_s(t1 - t0 == 1);
        for (int t = t0 + 1; t < t1 && ok; t++) {
          issue_s(t == t1 - 1);
          if (ok) issue_pv(t - 1 == t0);
        }
        if (ok) issue_pv(t1 - t0 == 1);
        qc++;
        pos.next(a);
      }
      if (!ok) sm.failed = 1;
    }
    __syncwarp();
  } else if (warp < nsw) {
    // --------------------------------------------------------- softmax
    constexpr int NB = CW / 8;       // 8-row blocks of this warpgroup's rows
    constexpr bool kKeep = CW == 32;  // both halves' exponents fit the registers between the passes
    const int wg = warp >> 2, quarter = warp & 3;
    const int c0 = wg * CW;          // this warpgroup's first row
    const int bar = 1 + wg, wt = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int key = quarter * 32 + lane;
    float *nb = sm.nb + c0;
    float *scr = reinterpret_cast<float *>(CW == 32 ? base + kTtHead + wg * (24 * CW)
                                               : base + at.p + c0 * 128);
    const float zs = a.zscale;
    const int64_t n_blocks = a.n_slots / a.BS;
    // stmatrix (transposing): matrices (keys 0–7 | 8–15) × (block k | k + 1);
    // this lane's query row of block 0, and its chunk of eight keys
    const int mrow = c0 + (lane >> 4) * 8 + (lane & 7);
    const int mchunk = quarter * 4 + ((lane >> 3) & 1);
    uint32_t sc = 0, qc = 0;  // tiles and runs done
    while (pos.g < pos.run1 && ok) {
      const int t0 = pos.t0, t1 = pos.t1(), h = pos.h(), rt = pos.rt(), n_rows = pos.rows(a);
      const int cols = max(0, min(CW, n_rows - c0));  // this warpgroup's rows of the run
      const int32_t *bt = a.block_table + (int64_t)pos.r * a.max_blocks;
      const int end = pos.c + pos.T;
      named_sync(bar, 128);                           // the last run's references are read
      if (wt < CW && c0 + wt < a.rows) nb[wt] = -kUnset;
      // −reference and sum of weights of rows 8k + 2·(t%4) + {0, 1}, and the
      // greatest −reference of them
      float nbr[2 * NB], l[2 * NB], nb_top = -kUnset;
#pragma unroll
      for (int e = 0; e < 2 * NB; e++) {
        nbr[e] = 8 * (e >> 1) + 2 * (lane & 3) + (e & 1) < cols ? -kUnset : -INFINITY;
        l[e] = 0.f;
      }
      // A wait that gives up only clears this warp's `ok`; the warpgroup leaves
      // together, at the next vote.
      for (int t = t0; t < t1; t++, sc++) {
        const int b = sc % p.SB;
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.sfull + b),
                                                             (sc / p.SB) & 1, &sm.failed));
        tc_fence_after();
        // a tile with nodes, past the end, or (after some bad block) any tile
        uint32_t see[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        const bool masked = (t + 1) * kTtKeys > pos.c || sm.bad;
        if (masked) {
          const int pp = t * kTtKeys + key;
          bool valid = pp < end;
          if (valid) {
            const int32_t blk = bt[pp / a.BS];
            valid = blk >= 0 && blk < n_blocks;
          }
          const uint32_t valid_keys = __ballot_sync(0xFFFFFFFFu, valid);
          see[0] = see[1] = 0;
#pragma unroll 1
          for (int e = 0; e < 8 * NB; e++) {
            const int hf = e / (4 * NB), k = (e >> 2) % NB, kk = hf * 16 + lane / 4 + 8 * ((e >> 1) & 1);
            const int x = c0 + 8 * k + 2 * (lane & 3) + (e & 1);
            const int j = t * kTtKeys + quarter * 32 + kk - pos.c, i = (rt * a.rstep + x) / a.G;
            bool v = (valid_keys >> kk) & 1u;
            if (v && j >= 0)
              v = i < pos.T &&
                  (a.mask ? (a.mask[(int64_t)(pos.q0 + i) * a.mask_words + (j >> 5)] >> (j & 31)) & 1u
                          : j <= i);
            const uint32_t bit = (uint32_t)v << (e % (4 * NB));
            if (hf == 0) see[0] |= bit;
            else see[1] |= bit;
          }
        }
        const uint32_t ts = tmem + lanes + b * a.rows + c0;
        // Pass 1: does some logit pass its row's reference by too much?  The
        // greatest logit against the least reference answers for almost every
        // tile; a tile that this does not clear is looked at row by row.
        float top = -INFINITY;
        uint32_t z[kKeep ? 2 : 1][4 * NB];
        if (ok && cols > 0) {
          if constexpr (kKeep) {
            tmem_frag<NB>(ts, z[0]);
            tmem_frag<NB>(ts + (16u << 16), z[1]);
            tmem_wait(z[0]);
            tmem_wait(z[1]);
#pragma unroll
            for (int e = 0; e < 4 * NB; e++)
              top = max3(top, __uint_as_float(z[0][e]), __uint_as_float(z[kKeep][e]));
          } else {
#pragma unroll 1
            for (int hf = 0; hf < 2; hf++) {
              tmem_frag<NB>(ts + ((uint32_t)(16 * hf) << 16), z[0]);
              tmem_wait(z[0]);
#pragma unroll
              for (int e = 0; e < 4 * NB; e += 2)
                top = max3(top, __uint_as_float(z[0][e]), __uint_as_float(z[0][e + 1]));
            }
          }
          top = fmaf(top, zs, nb_top);
          if (masked || zs < 0.f || __any_sync(0xFFFFFFFFu, !(top <= kExceed))) {
            top = -INFINITY;
#pragma unroll 1
            for (int hf = 0; hf < 2; hf++) {
              uint32_t y[4 * NB];
              float x[4 * NB];
              tmem_frag<NB>(ts + ((uint32_t)(16 * hf) << 16), y);
              tmem_wait(y);
              tree_exponents<NB>(y, zs, nbr, masked, see[hf], x);
#pragma unroll
              for (int e = 0; e < 4 * NB; e += 2) top = max3(top, x[e], x[e + 1]);
            }
          }
        }
        // the vote also keeps the warpgroup's warps within one tile of each other
        const bool raise = named_sync_or(bar, 128, !ok || top > kExceed);
        if (raise) {
          const uint32_t pv = sc - 1;  // the product before this tile's
          if (sc > 0 && ok)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.pvdone + (pv & 1)),
                                                           (pv >> 1) & 1, &sm.failed));
          // (every product that reads P is done: its memory may serve as scratch)
          ok = named_sync_and(bar, 128, ok);
          if (!ok) break;
          {
            float cm[2 * NB];
#pragma unroll
            for (int e = 0; e < 2 * NB; e++) cm[e] = -INFINITY;
            float zero[2 * NB];
#pragma unroll
            for (int e = 0; e < 2 * NB; e++) zero[e] = 0.f;
#pragma unroll 1
            for (int hf = 0; hf < 2; hf++) {
              uint32_t y[4 * NB];
              float x[4 * NB];
              tmem_frag<NB>(ts + ((uint32_t)(16 * hf) << 16), y);
              tmem_wait(y);
              tree_exponents<NB>(y, zs, zero, masked, see[hf], x);
#pragma unroll
              for (int k = 0; k < NB; k++) {
                cm[2 * k] = max3(cm[2 * k], x[4 * k], x[4 * k + 2]);
                cm[2 * k + 1] = max3(cm[2 * k + 1], x[4 * k + 1], x[4 * k + 3]);
              }
            }
#pragma unroll
            for (int e = 0; e < 2 * NB; e++) {
#pragma unroll
              for (int o = 4; o < 32; o <<= 1)
                cm[e] = fmaxf(cm[e], __shfl_xor_sync(0xFFFFFFFFu, cm[e], o));
              if (lane < 4) scr[quarter * CW + (e >> 1) * 8 + 2 * lane + (e & 1)] = cm[e];
            }
          }
          named_sync(bar, 128);
          if (wt < cols) {
            const float was = -nb[wt];
            const float m = fmaxf(fmaxf(scr[wt], scr[CW + wt]), fmaxf(scr[2 * CW + wt], scr[3 * CW + wt]));
            const float now = fmaxf(was, m);
            scr[4 * CW + wt] = ex2(was - now);
            nb[wt] = -now;
          }
          named_sync(bar, 128);
          const float *fac = scr + 4 * CW;
          nb_top = -INFINITY;
#pragma unroll
          for (int e = 0; e < 2 * NB; e++) {
            const int x = 8 * (e >> 1) + 2 * (lane & 3) + (e & 1);
            if (x < cols) {
              l[e] *= fac[x];
              nbr[e] = nb[x];
              nb_top = fmaxf(nb_top, nbr[e]);
            }
          }
          if (t > t0) {
#pragma unroll 1
            for (int cc = 0; cc < cols; cc += 16) {
              float v[16];
              tmem_ld16(tmem_o + lanes + c0 + cc, v);
#pragma unroll
              for (int e = 0; e < 16; e++)
                if (cc + e < cols) v[e] *= fac[cc + e];
              tmem_st16(tmem_o + lanes + c0 + cc, v);
            }
          }
          named_sync(bar, 128);  // the factors are read before P replaces them
        } else if (sc >= (uint32_t)p.PB) {
          const uint32_t u = sc - p.PB;  // P's buffer is free
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.pvdone + (u & 1)), (u >> 1) & 1,
                                                         &sm.failed));
        }
        // pass 2: the weights
        if (ok) {
          const uint32_t pbase = (base_u + at.p) + (sc % p.PB) * p_bytes;
          auto weights = [&](int hf, const uint32_t (&zz)[4 * NB]) {
            float w[4 * NB];
            tree_exponents<NB>(zz, zs, nbr, masked, see[hf], w);
#pragma unroll
            for (int e = 0; e < 4 * NB; e++) w[e] = ex2(w[e]);
#pragma unroll
            for (int k = 0; k < NB; k++) {
              l[2 * k] += w[4 * k] + w[4 * k + 2];
              l[2 * k + 1] += w[4 * k + 1] + w[4 * k + 3];
            }
            const int ch = mchunk + hf * 2;
            const uint32_t pa = pbase + (ch >> 3) * (a.rows * 128) + mrow * 128 +
                                (((ch & 7) ^ (mrow & 7)) << 4);
#pragma unroll
            for (int k = 0; k < NB; k += 2)
              if (8 * k < cols)
                stsm4t(pa + k * 1024,
                       pack_bf16x2(w[4 * k], w[4 * k + 1]), pack_bf16x2(w[4 * k + 2], w[4 * k + 3]),
                       pack_bf16x2(w[4 * k + 4], w[4 * k + 5]), pack_bf16x2(w[4 * k + 6], w[4 * k + 7]));
          };
          if constexpr (kKeep) {
            weights(0, z[0]);
            weights(1, z[kKeep]);
          } else {
#pragma unroll 1
            for (int hf = 0; hf < 2; hf++) {
              tmem_frag<NB>(ts + ((uint32_t)(16 * hf) << 16), z[0]);
              tmem_wait(z[0]);
              weights(hf, z[0]);
            }
          }
        } else {
          sm.failed = 1;
        }
        tc_fence_before();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(sm.sfree + b));
          mbar_arrive(smem_u32(sm.pready + (sc & 1)));
        }
      }
      // ---- the run's result: sums over the key lanes, then O
      const uint32_t pv = sc - 1;
      if (ok)
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.pvdone + (pv & 1)), (pv >> 1) & 1,
                                                       &sm.failed));
      ok = named_sync_and(bar, 128, ok);
      if (!ok) break;
      tc_fence_after();
      // (P is free: its last product is done)
#pragma unroll
      for (int e = 0; e < 2 * NB; e++) {
        float x = l[e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        if (lane < 4) scr[quarter * CW + 8 * (e >> 1) + 2 * lane + (e & 1)] = x;
      }
      named_sync(bar, 128);
      const bool whole = t0 == 0 && t1 == pos.n_kt;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (pos.g != pos.run0);
      if (wt < cols) {
        const float sum = (scr[wt] + scr[CW + wt]) + (scr[2 * CW + wt] + scr[3 * CW + wt]);
        const float m = sum > 0.f || sum != sum ? -nb[wt] : -INFINITY;
        const int x = rt * a.rstep + c0 + wt;
        if (whole) {
          const int64_t qr = (int64_t)(pos.q0 + x / a.G) * a.Hq + h * a.G + x % a.G;
          a.lse[qr] = m == -INFINITY ? -INFINITY : (m + log2f(sum)) * kLn2;
        } else {
          a.part_ml[slot * a.rows + c0 + wt] = make_float2(m, sum);
        }
        scr[4 * CW + wt] = whole ? (m == -INFINITY ? 0.f : 1.f / sum) : 1.f;
      }
      named_sync(bar, 128);
      const float *fac = scr + 4 * CW;
      const int d = D == 64 ? key & 63 : key;
      const bool odd = sm.odd != 0;
#pragma unroll 1
      for (int cc = 0; cc < cols; cc += 16) {
        float v[16];
        tmem_ld16(tmem_o + lanes + c0 + cc, v);
        if (odd) {  // infinities and NaN of the nodes this run covered, to the rows that see them
#pragma unroll 1
          for (int jn = max(0, t0 * kTtKeys - pos.c); jn < min(pos.T, t1 * kTtKeys - pos.c); jn++) {
            const int pn = pos.c + jn;
            const int32_t bn = bt[pn / a.BS];
            if (bn < 0 || bn >= n_blocks) continue;
            const float vn = bf16_lo(a.vpool[(((int64_t)bn * a.BS + pn % a.BS) * a.H + h) * D + d]);
            if (fabsf(vn) < INFINITY) continue;
#pragma unroll
            for (int e = 0; e < 16; e++) {
              const int i = (rt * a.rstep + c0 + cc + e) / a.G;
              if (i >= pos.T) continue;
              const bool see = a.mask ? (a.mask[(int64_t)(pos.q0 + i) * a.mask_words + (jn >> 5)] >> (jn & 31)) & 1u
                                      : jn <= i;
              if (see) v[e] += vn;
            }
          }
        }
        if (D == 64 && key >= 64) continue;  // (the second copy of V)
        if (whole) {
          int x = rt * a.rstep + c0 + cc, i = x / a.G, gg = x % a.G;
          uint16_t *o = a.out + ((int64_t)(pos.q0 + i) * a.Hq + h * a.G + gg) * D + d;
#pragma unroll
          for (int e = 0; e < 16; e++) {
            if (cc + e < cols) {
              const float f = fac[cc + e];
              const __nv_bfloat16 ob = __float2bfloat16(f == 0.f ? 0.f : v[e] * f);
              *o = *reinterpret_cast<const uint16_t *>(&ob);
              o += D;
              if (++gg == a.G) {
                gg = 0;
                o += (int64_t)(a.Hq - a.G) * D;
              }
            }
          }
        } else {
          float *o = a.part_o + (slot * a.rows + c0 + cc) * D + d;
#pragma unroll
          for (int e = 0; e < 16; e++)
            if (cc + e < cols) o[e * D] = v[e];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.ofree));
      qc++;
      pos.next(a);
    }
    if (!ok) {
      sm.failed = 1;
      if (lane == 0) record_error(a.status, KVC_ERR_TIMEOUT);
    }
  }

  // -------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (sm.failed && tid == 0) {
    record_error(a.status, KVC_ERR_TIMEOUT);
    // let this CTA's copies and products finish before its memory is released
    for (int i = 0; i < p.NS; i++) {
      mbar_drain(smem_u32(sm.full + i), 0);
      mbar_drain(smem_u32(sm.full + i), 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_drain(smem_u32(sm.sfull + i), 0);
      mbar_drain(smem_u32(sm.sfull + i), 1);
      mbar_drain(smem_u32(sm.pvdone + i), 0);
      mbar_drain(smem_u32(sm.pvdone + i), 1);
    }
  }
  __syncthreads();
  if (warp == nsw + kTtProd) {
    tc_fence_after();
    free_tmem_cols(tmem, 512);
  }
}

// Joins the partials of one (request, KV head, row tile) that was split over
// CTAs: blockIdx.x = (request, KV head), blockIdx.y = row tile, blockIdx.z a
// group of four rows.
template <int D>
__global__ void __launch_bounds__(128)
k_tree_join(TreeArgs a) {
  __shared__ int64_t sh[66];
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, rt = blockIdx.y;
  int64_t before = 0, total = 0;
  for (int x = threadIdx.x; x < a.n_req; x += blockDim.x) {
    const int64_t n = request_tiles(a, x);
    total += n;
    if (x < r) before += n;
  }
  before = block_sum(before, sh);
  total = block_sum(total, sh);
  int n_rt, n_kt;
  tree_tiles(a, r, n_rt, n_kt);
  // in every CTA: the grid may not end before the kernel whose partials it joins
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (rt >= n_rt) return;
  const int64_t g0 = before + ((int64_t)h * n_rt + rt) * n_kt;
  const int n_cta = (int)min((int64_t)a.n_cta, total);
  const int c0 = run_owner(total, n_cta, g0), c1 = run_owner(total, n_cta, g0 + n_kt - 1);
  if (c0 == c1) return;  // written whole
  int c, q0, T;
  tree_request(a, r, c, q0, T);
  const int row = blockIdx.z * 4 + threadIdx.x / 32, x = rt * a.rstep + row;
  if (row >= a.rstep || x >= T * a.G) return;
  const int64_t first = 2 * (int64_t)c0 + (run_start(total, n_cta, c0) != g0);
  const int n_part = c1 - c0 + 1;
  // part i is slot first (i = 0) or 2·(c0 + i): later CTAs begin inside the unit
  float mx = -INFINITY;
  for (int i = threadIdx.x & 31; i < n_part; i += 32)
    mx = fmaxf(mx, a.part_ml[(i == 0 ? first : 2 * (int64_t)(c0 + i)) * a.rows + row].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  const float base = mx == -INFINITY ? 0.f : mx;
  constexpr int E = D / 32;
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = 0.f;
  const int d0 = (threadIdx.x & 31) * E;
#pragma unroll 4
  for (int i = 0; i < n_part; i++) {
    const int64_t at = (i == 0 ? first : 2 * (int64_t)(c0 + i)) * a.rows + row;
    const float2 ml = a.part_ml[at];
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - base);
    sum = fmaf(ml.y, f, sum);
    float v[E];
    if constexpr (E == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(a.part_o + at * D + d0);
    else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(a.part_o + at * D + d0);
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] = fmaf(v[e], f, acc[e]);
  }
  const float inv = mx == -INFINITY ? 0.f : 1.f / sum;
  const int64_t qr = (int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G;
  uint32_t w[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; e++) w[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if constexpr (E == 4) *reinterpret_cast<uint2 *>(a.out + qr * D + d0) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t *>(a.out + qr * D + d0) = w[0];
  if (d0 == 0) a.lse[qr] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

// Rows up to which the narrow instruction is used.
constexpr int kRowsMax = 32;
constexpr int kTcRowsMax = 256;

// Rows per tile, keys per tile and grid of a call.
void tree_plan(int n_req, int max_blocks, int max_tree, int H, int Hq, int D, int BS, int &rows,
               int &rstep, int &tile, int &n_cta, int &max_rt) {
  const int G = Hq / H, R = max_tree * G;
  const bool tc = R > kRowsMax;
  rows = tc ? std::min((R + 31) / 32 * 32, kTcRowsMax) : R <= 16 ? 16 : 32;
  tile = tc ? kTtKeys : kRowWarps * (2048 / D);
  rstep = tc ? std::min(max_tree, rows / G) * G : rows;
  max_rt = (R + rstep - 1) / rstep;
  const int64_t most =
      (int64_t)n_req * H * max_rt * (((int64_t)max_blocks * BS + tile - 1) / tile);
  n_cta = (int)std::min<int64_t>((tc ? 1 : 2) * device_sm_count(), most);
}

// Boxes of `box` consecutive slots of one head, 64 columns, 128-byte swizzle.
bool pool_map(CUtensorMap *m, const void *pool, int64_t n_slots, int H, int D, int box) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)n_slots};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
  cuuint32_t bx[3] = {64, 1, (cuuint32_t)box}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(pool), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes of `nodes` consecutive rows of q, the G heads of one group, 64 columns.
bool q_map(CUtensorMap *m, const void *q, int n_q, int Hq, int D, int G, int nodes) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)n_q};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2};
  cuuint32_t bx[3] = {64, (cuuint32_t)G, (cuuint32_t)nodes}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int CW>
cudaError_t launch_tc(const TreeArgs &a, cudaStream_t s) {
  constexpr size_t kSmemMax = 232448;
  TreeTc p;
  p.NW = (a.rows + CW - 1) / CW;
  p.PB = a.rows <= 128 ? 2 : 1;
  p.SB = 3 * a.rows <= 512 ? 2 : 1;
  for (p.NS = kTtSlots; p.NS > 3; p.NS--)
    if (1024 + TreeTcSmem(D, a.rows, p.NS, p.PB).bytes <= kSmemMax) break;
  CUtensorMap tm_k{}, tm_v{}, tm_q{};
  p.box = a.BS % 32 == 0 ? 32 : a.BS % 16 == 0 ? 16 : a.BS % 8 == 0 ? 8 : 0;
  if (p.box && !(pool_map(&tm_k, a.kpool, a.n_slots, a.H, D, p.box) &&
                 pool_map(&tm_v, a.vpool, a.n_slots, a.H, D, p.box)))
    return cudaErrorUnknown;
  p.q_nodes = a.rstep / a.G;
  if (!q_map(&tm_q, a.q, a.n_q, a.Hq, D, a.G, p.q_nodes)) return cudaErrorUnknown;
  p.idesc_s = make_idesc(128, 0);
  p.idesc_o = make_idesc(128, 0) | (1u << 15);  // A (V) MN-major
  const size_t smem = 1024 + TreeTcSmem(D, a.rows, p.NS, p.PB).bytes;
  cudaError_t e = cudaFuncSetAttribute(k_tree_tc<D, CW>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k_tree_tc<D, CW><<<a.n_cta, (p.NW * 4 + kTtProd + 1) * 32, smem, s>>>(tm_k, tm_v, tm_q, a, p);
  return cudaGetLastError();
}

template <int D, int MT>
cudaError_t launch_rows(const TreeArgs &a, cudaStream_t s) {
  constexpr int smem = RowSmem<D, MT>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(k_tree_rows<D, MT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_tree_rows<D, MT><<<a.n_cta, kRowThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t tree_attn_ws_bytes(int n_req, int max_blocks, int max_tree, int H, int Hq, int D, int BS) {
  int rows, rstep, tile, n_cta, max_rt;
  tree_plan(n_req, max_blocks, max_tree, H, Hq, D, BS, rows, rstep, tile, n_cta, max_rt);
  return (size_t)2 * n_cta * rows * (D * sizeof(float) + sizeof(float2));
}

cudaError_t launch_tree_attn(const uint16_t *q, const uint16_t *kpool, const uint16_t *vpool,
                             int64_t n_slots, const int32_t *block_table, int max_blocks,
                             const int32_t *ctx_len, const int32_t *q_off,
                             const uint32_t *tree_mask, int mask_words, int n_req, int n_q,
                             int max_tree, int H, int Hq, int D, int BS, float scale,
                             uint16_t *out, float *lse, void *ws, int32_t *status,
                             cudaStream_t s) {
  TreeArgs a{};
  a.q = q;
  a.kpool = kpool;
  a.vpool = vpool;
  a.block_table = block_table;
  a.ctx_len = ctx_len;
  a.q_off = q_off;
  a.mask = tree_mask;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.n_slots = n_slots;
  a.max_blocks = max_blocks;
  a.mask_words = mask_words;
  a.n_req = n_req;
  a.n_q = n_q;
  a.max_tree = max_tree;
  a.H = H;
  a.Hq = Hq;
  a.G = Hq / H;
  a.BS = BS;
  a.zscale = scale * kLog2e;
  int max_rt;
  tree_plan(n_req, max_blocks, max_tree, H, Hq, D, BS, a.rows, a.rstep, a.tile, a.n_cta, max_rt);
  a.part_o = reinterpret_cast<float *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)2 * a.n_cta * a.rows * D);
  cudaError_t e;
  if (a.tile == kTtKeys && max_tree * a.G > kRowsMax)
    e = D == 128 ? (a.rows <= 128 ? launch_tc<128, 32>(a, s) : launch_tc<128, 64>(a, s))
                 : (a.rows <= 128 ? launch_tc<64, 32>(a, s) : launch_tc<64, 64>(a, s));
  else
    e = D == 128 ? (a.rows == 16 ? launch_rows<128, 1>(a, s) : launch_rows<128, 2>(a, s))
                 : (a.rows == 16 ? launch_rows<64, 1>(a, s) : launch_rows<64, 2>(a, s));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)n_req * H), (unsigned)max_rt, (unsigned)(a.rows / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return D == 128 ? cudaLaunchKernelEx(&cfg, k_tree_join<128>, a)
                  : cudaLaunchKernelEx(&cfg, k_tree_join<64>, a);
}

}  // namespace kvc
