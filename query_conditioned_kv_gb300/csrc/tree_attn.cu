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
  int rows;      // rows per row tile
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
  n_rt = (T * a.G + a.rows - 1) / a.rows;
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
    const int n_rows = min(R, T * a.G - rt * R);
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
      const int row = e / CH, col = e % CH, x = rt * R + row;
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
            const int x = rt * R + mt * 16 + hf * 8 + lane / 4;
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
        const int x = rt * R + row;
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
  const int row = blockIdx.z * 4 + threadIdx.x / 32, x = rt * a.rows + row;
  if (row >= a.rows || x >= T * a.G) return;
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

// Rows per tile, keys per tile and grid of a call.
void tree_plan(int n_req, int max_blocks, int max_tree, int H, int Hq, int D, int BS, int &rows,
               int &tile, int &n_cta, int &max_rt) {
  const int R = max_tree * (Hq / H);
  rows = R <= 16 ? 16 : 32;
  tile = kRowWarps * (2048 / D);
  max_rt = (R + rows - 1) / rows;
  const int64_t most =
      (int64_t)n_req * H * max_rt * (((int64_t)max_blocks * BS + tile - 1) / tile);
  n_cta = (int)std::min<int64_t>(2 * device_sm_count(), most);
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
  int rows, tile, n_cta, max_rt;
  tree_plan(n_req, max_blocks, max_tree, H, Hq, D, BS, rows, tile, n_cta, max_rt);
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
  tree_plan(n_req, max_blocks, max_tree, H, Hq, D, BS, a.rows, a.tile, a.n_cta, max_rt);
  a.part_o = reinterpret_cast<float *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)2 * a.n_cta * a.rows * D);
  cudaError_t e = D == 128 ? (a.rows == 16 ? launch_rows<128, 1>(a, s) : launch_rows<128, 2>(a, s))
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
