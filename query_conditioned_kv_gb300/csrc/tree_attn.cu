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
// does not depend on timing.  Where requests are short, a cluster of up to 16
// CTAs takes a unit instead and joins its parts from one another's shared
// memory: one launch, and no search for the run (tree_cluster says when).
//
// k_tree_rows (up to 32 rows a tile): each of a CTA's four warps streams its
// own quarter of every tile through a private cp.async ring (3 stages of
// 8 KB, so about 128 KB in flight per SM with two CTAs) and keeps its own
// softmax statistics and accumulators; no barrier until the run ends.  The
// products are mma.sync m16n8k16 with fp32 accumulators: at 16 rows the
// tensor work per key is a few per cent of the time its bytes take, so the
// narrow instruction, which needs no shared-memory round trip for the
// weights, is enough.  Measured: one token of 64 requests, 4K to 8K, 8 KV heads,
// D 128: 250 us, 6.45 TB/s, 96 % of a plain copy's rate; one request of 4K 12 us,
// of which launch and the chain sizes → block ids → rows → join are all but 3.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "kvc_internal.cuh"
#include "tree_rows.cuh"

namespace kvc {
namespace {

using namespace tc;

constexpr int kRowWarps = 4;
constexpr int kRowThreads = kRowWarps * 32;
constexpr int kRowStages = 3;
constexpr int kWarpStage = 8192;  // bytes of one warp's stage: K rows, then V rows

template <int D, int MT>
struct RowSmem {
  static constexpr int kRing = kRowWarps * kRowStages * kWarpStage;
  static constexpr int kQ = kRing;                       // MT·16 rows of q
  static constexpr int kValid = kQ + MT * 16 * D * 2;  // valid keys per (warp, stage)
  static constexpr int kMl = kValid + kRowWarps * kRowStages * 4;  // (max, sum) per (warp, row)
  static constexpr int kClMl = kMl + kRowWarps * MT * 16 * 8;      // (max, sum) of the CTA, per row
  static constexpr int kBytes = kClMl + MT * 16 * 8;
  static constexpr int kClO = kRowWarps * MT * 16 * D * 4;  // the CTA's O, behind the warps'
  static_assert(kClO + MT * 16 * D * 4 <= kRing, "the warps' and the CTA's O fit the ring");
};

// O += W·V for the KT keys of a warp's tile (V rows at vb, the first key's position
// p0), weights in the score registers of MT row tiles of 16.
template <int D, int MT, int KT>
__device__ __forceinline__ void tile_values(const TreeArgs &a, const float (&s)[MT][KT / 8][4],
                                            float (&o)[MT][D / 8][4], uint32_t vb, uint32_t okb,
                                            int rt, int q0, int c, int T, int p0) {
  constexpr int NT = D / 8, CH = D / 8;
  const int lane = threadIdx.x & 31;
  // A node's V may hold infinities or NaN that some rows do not see, and a
  // product 0·inf would hand them to those rows.  A tile with such values
  // takes the sum term by term, over the rows' visible keys only; there such a
  // value is added as it is, for a weight too small for fp32 is not 0.
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
    auto add = [](float w, float v, float &acc) {
      acc = fabsf(v) < INFINITY ? fmaf(w, v, acc) : acc + v;
    };
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      uint32_t vis[2];
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        const int x = rt * a.rstep + mt * 16 + hf * 8 + lane / 4;
        vis[hf] = x < T * a.G ? visible_bits<KT>(a, x / a.G, q0, c, T, p0) & okb : 0u;
      }
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
              if ((vis[0] >> (8 * kn + 2 * kq + e)) & 1u) {
                add(w0, bf16_lo(v), o[mt][n][0]);
                add(w0, bf16_hi(v), o[mt][n][1]);
              }
              if ((vis[1] >> (8 * kn + 2 * kq + e)) & 1u) {
                add(w1, bf16_lo(v), o[mt][n][2]);
                add(w1, bf16_hi(v), o[mt][n][3]);
              }
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
}

template <int D, int MT, bool CL>
__global__ void __launch_bounds__(kRowThreads, 2)
k_tree_rows(TreeArgs a) {
  using S = RowSmem<D, MT>;
  constexpr int KT = 2048 / D, KS = D / 16, NT = D / 8, CH = D / 8;
  constexpr int R = MT * 16;
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(sm) + warp * kRowStages * kWarpStage;
  uint32_t *valid_s = reinterpret_cast<uint32_t *>(sm + S::kValid) + warp * kRowStages;
  const uint32_t qbase = smem_u32(sm + S::kQ);
  float2 *ml_s = reinterpret_cast<float2 *>(sm + S::kMl);

  int r, c, q0, T, n_rt, n_kt, unit, t0;
  int64_t g, run0, run1;  // next tile of the run, its begin and end
  if constexpr (CL) {
    const int S = (int)cluster_nrank(), rank = (int)cluster_rank(), u = blockIdx.x / S;
    r = u / a.H;
    unit = u % a.H;
    const bool valid = tree_request(a, r, c, q0, T);
    if (!valid && unit == 0 && rank == 0 && tid == 0) record_error(a.status, KVC_ERR_BOUNDS);
    tree_tiles(a, r, n_rt, n_kt);
    if (n_rt == 0) return;  // (the whole cluster)
    t0 = n_kt * rank / S;
    g = run0 = 0;
    run1 = n_kt * (rank + 1) / S - t0;
  } else {
    asm volatile("griddepcontrol.launch_dependents;");
    if (blockIdx.x == 0)  // one report per bad request
      for (int r = tid; r < a.n_req; r += kRowThreads) {
        int c, q0, T;
        if (!tree_request(a, r, c, q0, T)) record_error(a.status, KVC_ERR_BOUNDS);
      }
    auto tiles = [&](int x) { return request_tiles(a, x); };
    const WarpSums sums = warp_sums(a.n_req, tiles);
    const int64_t total = sums.total;
    int64_t before;
    const int n_cta = (int)min((int64_t)a.n_cta, total);  // every run holds a tile
    if ((int)blockIdx.x >= n_cta) return;
    run0 = g = run_start(total, n_cta, blockIdx.x);
    run1 = run_start(total, n_cta, blockIdx.x + 1);
    warp_find(sums, a.n_req, run0, tiles, r, before);
    tree_request(a, r, c, q0, T);
    tree_tiles(a, r, n_rt, n_kt);
    unit = (int)div64(g - before, n_kt);  // h·n_rt + row tile
    t0 = (int)(g - before - (int64_t)unit * n_kt);
  }
  const int64_t n_blocks = a.n_slots / a.BS;
  while (CL || g < run1) {
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
        const int32_t b = bt[page_of(p, a.bs_inv)];
        if (b >= 0 && b < n_blocks) slot = b * a.BS + p - page_of(p, a.bs_inv) * a.BS;
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
      tile_values<D, MT, KT>(a, s, o, vb, okb, rt, q0, c, T, p0);
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
    const bool whole = !CL && t0 == 0 && t1 == n_kt;
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
        // This warp saw nothing of the row.  (Logits that are all NaN leave the
        // maximum at −inf too, but a NaN sum, which has to reach the result.)
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
        uint2 w2 = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2 *>(a.out + qr * D + d4) = w2;
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
      // the cluster's CTAs hold the unit's parts: added up in order, the elements
      // dealt out to all of them
      __syncwarp();
      cluster_sync_all();
      const int n_cl = (int)cluster_nrank();
      const uint32_t o_at = smem_u32(sm + S::kClO), ml_at = smem_u32(sm + S::kClMl);
      for (int e = (int)cluster_rank() * kRowThreads + tid; e < n_rows * (D / 4);
           e += n_cl * kRowThreads) {
        const int row = e / (D / 4), d4 = (e % (D / 4)) * 4;
        float mx = -INFINITY;
#pragma unroll 4
        for (int k = 0; k < n_cl; k++) mx = fmaxf(mx, ld_cluster_f2(mapa_u32(ml_at + row * 8, k)).x);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < n_cl; k++) {
          const float2 ml = ld_cluster_f2(mapa_u32(ml_at + row * 8, k));
          const float4 v = ld_cluster_f4(mapa_u32(o_at + (row * D + d4) * 4, k));
          const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx);
          sum = fmaf(ml.y, f, sum);
          acc.x = fmaf(v.x, f, acc.x);
          acc.y = fmaf(v.y, f, acc.y);
          acc.z = fmaf(v.z, f, acc.z);
          acc.w = fmaf(v.w, f, acc.w);
        }
        const int x = rt * a.rstep + row;
        const int64_t qr = (int64_t)(q0 + x / a.G) * a.Hq + h * a.G + x % a.G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2 *>(a.out + qr * D + d4) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (d4 == 0) a.lse[qr] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
      }
      __syncwarp();
      cluster_sync_all();  // (no CTA leaves while another reads its part)
      return;
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
// k_tree_tc (more than 32 rows).  Per job, 128 keys and up to 128 rows:
//   Sᵀ[key][row] = K·Qᵀ     (M 128 keys, N rows, K D; both K-major)
//   O[row][d]  += P·V       (M 128 rows, N D, K 128 keys; V as it lies in the
//                            pool, MN-major; P written K-major)
// Two softmax warpgroups (teams) take the jobs in turn, each with its own Sᵀ,
// P and O, so that one team's softmax runs under the other's
// products: at most 128 rows, a job is a tile and the teams' results are
// joined when the run ends; with more rows each tile is two jobs, team 0
// taking rows 0–127 and team 1 the others.
//
// A softmax thread owns four keys and 32 rows of a job (16x256b fragments),
// so a row's maximum is spread over a warpgroup.  The exponent's reference is
// therefore not the running maximum but a fixed value per row, the maximum of
// the team's first tile, raised only when some logit exceeds it by 2^30:
// weights, their sums and O stay far inside fp32 and bf16 range (bf16 has
// fp32's exponents), and the result does not depend on the reference.  A job
// is worked out on the references at hand; a vote of the warpgroup (one
// barrier) then passes it on, or raises the references, rescales O in tensor
// memory and works the job out again.  Once is enough: the reference is the largest
// rounded product S·zscale, and a logit taken as fma(S, zscale, −reference) passes
// it, or the largest falls short of it, by half a step of the reference at most:
// less than 1 below 2^24.  From there on (kRoundFrom) half a step may be hundreds.
// Then every job of the run raises the references first and writes the differences
// of the rounded products to them into Sᵀ, where the largest is 0.  A tile that
// holds nodes, or the end, first gets −inf written into Sᵀ where a row does not see
// a key, so the loop over the tiles has no masks.
//
// Warps: 0–7 softmax; 8–11 load K and V, 32 keys of a tile each (8 the queries
// too): TMA boxes of whole page rows, or cp.async row by row where a tile
// holds nodes, the end, or a page size has no box; 12 issues Sᵀ, 13 issues O.
// K and V share one ring of NS slots, filled in the order K0 K1 V0 K2 V1 …:
// with three slots (256 rows leave no room for more) a tile's K and V still
// have about a tile's time to arrive.  The barriers are per kind, not per
// slot: a barrier's parity tells only two uses apart, and two consumers of one
// ring may be further apart than that.
//
// Bound: with 128 rows the K and V stream (128K of one request, 109 us, 4.9
// TB/s); with 256 the products, about 105 cycles an instruction at N = 128 where
// N = 256 would take 126 (tensor memory holds S 256 + O 256 columns, so S of 256
// columns could not be worked on while the next is made): 64 nodes × 4 heads, 16
// requests of 16K to 32K, 412 to 443 us from one batch of trees to another, 700 to
// 750 TFLOP/s and 3.7 to 3.9 TB/s.  One stage at a time is in flight where a page has
// no box: 20 nodes × 4 heads, 4 requests of 32K, 167 us with pages of 5 or 12 and 118
// with pages of 16.

constexpr int kTtKeys = 128;
constexpr int kTtSoft = 8;
constexpr int kTtThreads = (kTtSoft + 8) * 32;  // (two warps fill the last warpgroup)
// Registers of a softmax thread, of the others (64 nodes, 16 requests: 420 us; 168
// and 88 423, 184 and 72 419 but 3 % slower with 128 rows, 160 and 96 426).
constexpr int kTtMore = 176, kTtLess = 80;
constexpr float kUnset = -FLT_MAX;  // reference of a row that has seen nothing
constexpr float kExceed = 30.f;    // log2 of how far a logit may pass the reference
constexpr float kRoundFrom = 16777216.f;  // |reference| from which Sᵀ gets rounded differences

struct TreeTc {
  int NS;      // ring slots: 3 or 4
  int box;     // rows of a TMA box (a divisor of the page size), 0: no TMA
  int q_nodes; // nodes of a row tile
  uint32_t idesc_s, idesc_o;  // idesc_s without N
};

constexpr int kTtSlots = 4;  // ring slots, at most; barriers of a kind

// Head of the dynamic shared memory, at fixed offsets (few live registers);
// then P of both teams, the ring and q.
struct TreeTcHead {
  uint64_t full[2][kTtSlots], empty[2][kTtSlots];  // [K, V][tile mod kTtSlots]
  uint64_t qfull, qempty;
  uint64_t sfull[2], sfree[2], pready[2], pvdone[2], ofree;  // [team]
  uint32_t tmem_holder;
  volatile int failed, odd;
  // Per team, what makes a job unlike the others: some bad block was met; a
  // reference of this run is past kRoundFrom.
  volatile union {
    uint16_t any;
    struct {
      uint8_t bad, large;
    };
  } special[2];
  float nb[2][128];  // −reference per team and row
};
constexpr uint32_t kTtHead = 2048;
static_assert(sizeof(TreeTcHead) <= kTtHead, "the head's room");
constexpr uint32_t kTtP = 128 * kTtKeys * 2;  // bytes of a team's P: [key half][row][64 keys]

// Byte offsets (multiples of 1024) from the head.
struct TreeTcSmem {
  uint32_t ring, q, bytes;
  __host__ __device__ TreeTcSmem(int D, int rows, int NS) {
    ring = kTtHead + 2 * kTtP;
    q = ring + NS * kTtKeys * D * 2;
    bytes = q + rows * D * 2;
  }
};

// Place of K tile t and V tile t of a run of nT tiles among its 2·nT stages.
__device__ __forceinline__ int stage_k(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int stage_v(int t, int nT) { return t < nT - 1 ? 2 * t + 2 : 2 * nT - 1; }

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
    unit = (int)div64(g - before, n_kt);
    t0 = (int)(g - before - (int64_t)unit * n_kt);
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

__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                      uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

// The same fragment written back.
__device__ __forceinline__ void tmem_put(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(kTtThreads, 1)
k_tree_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
          const __grid_constant__ CUtensorMap tm_q, TreeArgs a, TreeTc p) {
  constexpr int CH = D / 8, KB = D / 64;
  constexpr uint32_t kSlot = kTtKeys * D * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TreeTcHead &sm = *reinterpret_cast<TreeTcHead *>(base);
  const TreeTcSmem at(D, a.rows, p.NS);
  const uint32_t base_u = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) {
    sm.failed = 0;
    sm.odd = 0;
    sm.special[0].any = sm.special[1].any = 0;
    for (int i = 0; i < 2 * kTtSlots; i++) {
      mbar_init(smem_u32(sm.full[0] + i), 128);
      mbar_init(smem_u32(sm.empty[0] + i), 1);
    }
    mbar_init(smem_u32(&sm.qfull), 1);
    mbar_init(smem_u32(&sm.qempty), 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(smem_u32(sm.sfull + i), 1);
      mbar_init(smem_u32(sm.sfree + i), kTtSoft / 2);
      mbar_init(smem_u32(sm.pready + i), kTtSoft / 2);
      mbar_init(smem_u32(sm.pvdone + i), 1);
    }
    mbar_init(smem_u32(&sm.ofree), kTtSoft);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kTtSoft + 4) alloc_tmem_cols(&sm.tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_holder;  // Sᵀ of team 0, of team 1, O of team 0, of team 1

  if (blockIdx.x == 0)  // one report per bad request
    for (int r = tid; r < a.n_req; r += blockDim.x) {
      int c, q0, T;
      if (!tree_request(a, r, c, q0, T)) record_error(a.status, KVC_ERR_BOUNDS);
    }
  auto tiles = [&](int x) { return request_tiles(a, x); };
  const WarpSums sums = warp_sums(a.n_req, tiles);
  const int64_t total = sums.total;
  const int n_cta = (int)min((int64_t)a.n_cta, total);
  const bool works = (int)blockIdx.x < n_cta;
  TreePos pos{};
  if (works) {
    pos.run0 = pos.g = run_start(total, n_cta, blockIdx.x);
    pos.run1 = run_start(total, n_cta, blockIdx.x + 1);
    int64_t before;
    warp_find(sums, a.n_req, pos.g, tiles, pos.r, before);
    pos.init(a, before);
  }

  bool ok = true;
  // Registers move from the producers and MMA warps to the softmax: 256·kTtMore
  // + 256·kTtLess is the 512·128 of the launch.
  if (warp >= kTtSoft && warp < kTtSoft + 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTtLess));
    // ------------------------------------------------------- producers
    const int key0 = (warp & 3) * 32;  // this warp's keys of a tile
    const int64_t n_blocks = a.n_slots / a.BS;
    constexpr int RPI = 32 / CH;
    const int col = lane % CH;
    uint32_t rc = 0, qc = 0;            // stages filled, runs done
    uint32_t kc = 0, vc = 0;            // K tiles, V tiles filled
    uint32_t before[kTtSlots];          // what the last stages held: 2·tile + kind
#pragma unroll
    for (int i = 0; i < kTtSlots; i++) before[i] = 0;
    uint32_t pend = 0;  // a stage copied by cp.async and not yet handed over
    auto flush = [&]() {
      if (!pend) return;
      cp_wait<0>();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(pend);
      pend = 0;
    };
    // a full ring is waited for only after everything in flight is handed over
    auto acquire = [&](uint32_t bar, uint32_t parity) {
      if (mbar_try(bar, parity)) return true;
      flush();
      return mbar_wait_bounded(bar, parity, &sm.failed);
    };
    while (pos.g < pos.run1 && ok) {
      const int t0 = pos.t0, t1 = pos.t1(), h = pos.h(), rt = pos.rt();
      const int32_t *bt = a.block_table + (int64_t)pos.r * a.max_blocks;
      const int end = pos.c + pos.T;
      const uint32_t uh = uniform32(h);
      int32_t blk, slot = -1;  // block id of the next tile's key, slot of this tile's
      auto fetch = [&](int t) {
        const int pp = t * kTtKeys + key0 + lane;
        blk = pp < end && t < t1 ? bt[page_of(pp, a.bs_inv)] : 0;
      };
      auto resolve = [&](int t) {
        const int pp = t * kTtKeys + key0 + lane;
        slot = -1;
        if (pp < end) {
          if (blk >= 0 && blk < n_blocks) {
            slot = blk * a.BS + pp - page_of(pp, a.bs_inv) * a.BS;
          } else {
            // (read by the softmax warps after this stage's product)
            sm.special[0].bad = sm.special[1].bad = 1;
            record_error(a.status, KVC_ERR_BOUNDS);
          }
        }
      };
      // One stage: tile t of K or V, this warp's keys in `slot`.
      auto load = [&](int t, bool is_v, int32_t slot) {
        // the ring slot's last use has been consumed
        const uint32_t was = p.NS == 3 ? before[2] : before[3];
        if (rc >= (uint32_t)p.NS &&
            !(ok = acquire(smem_u32(sm.empty[was & 1] + (was >> 1) % kTtSlots),
                           ((was >> 1) / kTtSlots) & 1)))
          return;
        const uint32_t c = is_v ? vc++ : kc++;
#pragma unroll
        for (int i = kTtSlots - 1; i > 0; i--) before[i] = before[i - 1];
        before[0] = 2 * c + is_v;
        const uint32_t slot0 = base_u + at.ring + (rc % p.NS) * kSlot + key0 * 128;
        rc++;
        const uint32_t bar = smem_u32(sm.full[is_v] + c % kTtSlots);
        // TMA boxes of whole page rows where every key is cached, else row by
        // row with cp.async (zeros past the end)
        if (p.box > 0 && (t + 1) * kTtKeys <= pos.c && __all_sync(0xFFFFFFFFu, slot >= 0)) {
          if (lane == 0) mbar_expect_tx(bar, kSlot / 4);
          else mbar_arrive(bar);
          __syncwarp();
          // (warp-uniform operands, one lane enabled: see the MMA warps)
          const uint32_t ubar = uniform32(bar), udst = uniform32(slot0);
          const CUtensorMap *tm = is_v ? &tm_v : &tm_k;
          for (int k = 0; k < 32; k += p.box) {  // a box's first key
            const uint32_t sl = __shfl_sync(0xFFFFFFFFu, slot, k);
#pragma unroll
            for (int kb = 0; kb < KB; kb++)
              tma_load_3d_if(lane == 0, udst + k * 128 + kb * (kTtKeys * 128), tm, kb * 64, uh, sl, ubar);
          }
          return;
        }
        flush();
        const uint16_t *pool = is_v ? a.vpool : a.kpool;
        const uint32_t dst = slot0 + (col >> 3) * (kTtKeys * 128);
#pragma unroll 4
        for (int k = 0; k < 32 / RPI; k++) {
          const int row = k * RPI + lane / CH;
          const int32_t sl = __shfl_sync(0xFFFFFFFFu, slot, row);
          cp_async16(dst + row * 128 + (((col & 7) ^ (row & 7)) << 4),
                     pool + ((int64_t)max(sl, 0) * a.H + h) * D + col * 8, sl >= 0);
        }
        cp_commit();
        pend = bar;
        if (is_v && (t + 1) * kTtKeys > pos.c) {
          // A node's V may hold infinities or NaN that some rows do not see: the
          // product gets zeros in their place, and the run's end adds them to
          // the rows that do.  Each thread looks at what it copied, before the
          // stage is handed over.
          cp_wait<0>();
          bool odd = false;
#pragma unroll 1
          for (int k = 0; k < 32 / RPI; k++) {
            const int row = k * RPI + lane / CH;
            const uint32_t ad = dst + row * 128 + (((col & 7) ^ (row & 7)) << 4);
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(ad)
                         : "memory");
            bool mine = false;
#pragma unroll
            for (int u = 0; u < 4; u++) {
              if ((w[u] & 0x7F80u) == 0x7F80u) mine = true, w[u] &= 0xFFFF0000u;
              if ((w[u] & 0x7F800000u) == 0x7F800000u) mine = true, w[u] &= 0xFFFFu;
            }
            // (cached positions are seen by every row: their values stay)
            if (mine && t * kTtKeys + key0 + row >= pos.c) {
              odd = true;
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(ad), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
          if (odd) sm.odd = 1;
          flush();
        }
      };
      fetch(t0);
      for (int t = t0; t < t1 && ok; t++) {
        const int32_t slot_v = slot;  // of tile t − 1
        resolve(t);
        fetch(t + 1);
        load(t, false, slot);
        if (!ok) break;
        if (t == t0) {
          // the row tile's queries, in one box of nodes × heads of the group; rows
          // past the request's own (another request's, or zeros) are columns that
          // the softmax leaves out
          if (warp == kTtSoft) {
            if (!(ok = acquire(smem_u32(&sm.qempty), (qc & 1) ^ 1))) break;
            if (lane == 0) {
              const uint32_t qbar = smem_u32(&sm.qfull);
              mbar_expect_tx(qbar, p.q_nodes * a.G * D * 2);
#pragma unroll
              for (int kb = 0; kb < KB; kb++)
                tma_load_3d(base_u + at.q + kb * (a.rows * 128), &tm_q, kb * 64, h * a.G,
                            pos.q0 + rt * p.q_nodes, qbar);
            }
            __syncwarp();
          }
        } else {
          load(t - 1, true, slot_v);
        }
      }
      if (ok) load(t1 - 1, true, slot);
      qc++;
      pos.next(a);
    }
    flush();
    cp_wait<0>();
    if (!ok) sm.failed = 1;
  } else if (warp >= kTtSoft + 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTtLess));
    if (warp < kTtSoft + 6) {
    // ----------------------------------------------------- MMA issuers
    // One warp for each product: a warp stands still while its instructions
    // queue, and the tensor core would idle while it then waits for the other
    // product's operands.
    // The whole warp runs the loop and one lane's products are enabled by a
    // predicate: the descriptors then live in uniform registers.  (In a branch
    // of one lane every product cost some 100 cycles to issue.)
    const uint32_t lead = lane == 0;
    const bool first = warp == kTtSoft + 4;  // Sᵀ, or O
    uint32_t rc = 0, qc = 0;  // stages before this run, runs done
    uint32_t tc = 0;          // tiles used
    uint32_t done[2];         // jobs issued per team, by bit 0 (constant indexes only)
    done[0] = done[1] = 0;
    while (pos.g < pos.run1 && ok) {
      const int nT = pos.t1() - pos.t0, n_rows = pos.rows(a);
      const bool halves = n_rows > 128;
      if (first) {
        ok = mbar_wait_bounded(smem_u32(&sm.qfull), qc & 1, &sm.failed);
        const uint64_t qb = uniform64(smem_desc(base_u + at.q));
        const uint32_t qk = (uint32_t)a.rows * 8;  // next 64 columns of q, in 16 bytes
        const int nJ = halves ? 2 * nT : nT;
        for (int j = 0; j < nJ && ok; j++) {
          const int tm = j & 1, t = halves ? j >> 1 : j, row0 = halves ? 128 * tm : 0;
          const uint32_t st = tc % kTtSlots;
          ok = mbar_wait_bounded(smem_u32(sm.full[0] + st), (tc / kTtSlots) & 1, &sm.failed);
          if (ok)
            ok = mbar_wait_bounded(smem_u32(sm.sfree + tm), ((tm ? done[1] : done[0]) & 1) ^ 1,
                                   &sm.failed);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ka =
              uniform64(smem_desc(base_u + at.ring + ((rc + stage_k(t)) % p.NS) * kSlot));
          const uint32_t dst = uniform32(tmem + tm * 128);
          const uint32_t n8 = (min(n_rows - row0, 128) + 15) / 16 * 2;  // N / 8
          const uint32_t idesc = uniform32(p.idesc_s | (n8 << 17));
          const uint64_t qt = qb + uniform32(row0 * 8);
#pragma unroll
          for (int kk = 0; kk < 4 * KB; kk++)
            mma_bf16_if(lead, dst, ka + (kk >> 2) * (kTtKeys * 8) + (kk & 3) * 2,
                        qt + (kk >> 2) * qk + (kk & 3) * 2, idesc, kk > 0);
          mma_commit_if(lead, smem_u32(sm.sfull + tm));
          if (tm) done[1]++;
          else done[0]++;
          if (!halves || tm == 1) {
            mma_commit_if(lead, smem_u32(sm.empty[0] + st));
            tc++;
          }
          if (j == nJ - 1) mma_commit_if(lead, smem_u32(&sm.qempty));
        }
      } else {
        const int nJ = halves ? 2 * nT : nT;
        for (int j = 0; j < nJ && ok; j++) {
          const int tm = j & 1, t = halves ? j >> 1 : j;
          const uint32_t st = tc % kTtSlots;
          ok = mbar_wait_bounded(smem_u32(sm.full[1] + st), (tc / kTtSlots) & 1, &sm.failed);
          if (ok && j == 0)  // both O's previous contents have been read
            ok = mbar_wait_bounded(smem_u32(&sm.ofree), (qc & 1) ^ 1, &sm.failed);
          if (ok)
            ok = mbar_wait_bounded(smem_u32(sm.pready + tm), (tm ? done[1] : done[0]) & 1, &sm.failed);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vb = uniform64(smem_desc_mn(
              base_u + at.ring + ((rc + stage_v(t, nT)) % p.NS) * kSlot, kTtKeys * 128));
          const uint64_t pa = uniform64(smem_desc(base_u + kTtHead + tm * kTtP));
          const uint32_t dst = uniform32(tmem + 256 + tm * 128);
#pragma unroll
          for (int kk = 0; kk < kTtKeys / 16; kk++)
            mma_bf16_if(lead, dst, pa + (kk >> 2) * (kTtP / 32) + (kk & 3) * 2, vb + kk * 128, p.idesc_o,
                        j > 1 || kk > 0);
          mma_commit_if(lead, smem_u32(sm.pvdone + tm));
          if (tm) done[1]++;
          else done[0]++;
          if (!halves || tm == 1) {
            mma_commit_if(lead, smem_u32(sm.empty[1] + st));
            tc++;
          }
        }
      }
      rc += 2 * nT;
      qc++;
      pos.next(a);
    }
    if (!ok) sm.failed = 1;
    __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTtMore));
    // --------------------------------------------------------- softmax
    const int team = warp >> 2, quarter = warp & 3;
    const int bar = 1 + team, wt = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t ts = tmem + team * 128 + lanes, to = tmem + 256 + team * 128 + lanes;
    float *nb = sm.nb[team];
    uint8_t *p_team = base + kTtHead + team * kTtP;
    float *scr = reinterpret_cast<float *>(p_team);  // scratch while P is free
    const float zs = a.zscale;
    const int64_t n_blocks = a.n_slots / a.BS;
    // stmatrix (transposing): matrices (keys 0–7 | 8–15) × (8-row block k | k + 1);
    // this lane's row of block 0, and its chunk of eight keys
    const int mrow = (lane >> 4) * 8 + (lane & 7);
    const uint32_t pst = smem_u32(p_team) + (quarter >> 1) * (kTtP / 2) + mrow * 128;
    const int mchunk = (quarter & 1) * 4 + ((lane >> 3) & 1);
    uint32_t sc = 0;  // this team's jobs done
    while (pos.g < pos.run1 && ok) {
      const int t0 = pos.t0, t1 = pos.t1(), n_rows = pos.rows(a);
      const bool halves = n_rows > 128;
      const int row0 = halves ? team * 128 : 0;          // the team's first row
      const int cols = min(128, n_rows - row0);          // its rows
      const int32_t *bt = a.block_table + (int64_t)pos.r * a.max_blocks;
      named_sync(bar, 128);  // the last run's references are read
      nb[wt] = wt < cols ? -kUnset : -INFINITY;  // (columns that hold no row: weight 0)
      sm.special[team].large = 0;
      named_sync(bar, 128);
      // This thread's row's reference while they are large (in local memory: the loop
      // has no register to spare for it, 3 to 9 % of its time).
      volatile float large_ref[1];
      float l[32];  // sums of the weights of rows 8k + 2·(t%4) + {0, 1}
#pragma unroll
      for (int e = 0; e < 32; e++) l[e] = 0.f;
      // A wait that gives up only clears this warp's `ok`; the team leaves
      // together, at the next vote.
      bool fresh = true;
      for (int t = halves ? t0 : t0 + team; t < t1; t += halves ? 1 : 2, sc++) {
        ok = ok && __all_sync(0xFFFFFFFFu,
                              mbar_wait_bounded(smem_u32(sm.sfull + team), sc & 1, &sm.failed));
        tc_fence_after();
        // a tile with nodes, past the end, or (after some bad block, or with large
        // references) any tile
        if ((t + 1) * kTtKeys > pos.c || sm.special[team].any) {
          if (ok) {
            const int pp = t * kTtKeys + quarter * 32 + lane;
            bool valid = pp < pos.c + pos.T;
            if (valid) {
              const int32_t blk = bt[page_of(pp, a.bs_inv)];
              valid = blk >= 0 && blk < n_blocks;
            }
            const uint32_t valid_keys = __ballot_sync(0xFFFFFFFFu, valid);
            const float hidden = zs < 0.f ? INFINITY : -INFINITY;  // −inf once scaled
            // which of the warp's 32 keys the rows lane + 32·m see
            uint32_t sees[4];
            const int p0 = t * kTtKeys + quarter * 32, j0 = p0 - pos.c;
#pragma unroll
            for (int m = 0; m < 4; m++) {
              const int i = (pos.rt() * a.rstep + row0 + 32 * m + lane) / a.G;
              uint32_t v = j0 <= -32 ? 0xFFFFFFFFu : j0 < 0 ? (1u << -j0) - 1u : 0u;
              if (i < pos.T) v = visible_bits<32>(a, i, pos.q0, pos.c, pos.T, p0);
              sees[m] = v & valid_keys;
            }
#pragma unroll 1
            for (int ch = 0; ch < 2; ch++) {
              uint32_t bits[2] = {0, 0};  // of the registers of the two fragments (see tmem_frag8)
#pragma unroll
              for (int k = 0; k < 8; k++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                  const uint32_t mine = ch ? sees[2 + (k >> 2)] : sees[k >> 2];
                  const uint32_t v =
                      __shfl_sync(0xFFFFFFFFu, mine, 8 * (k & 3) + 2 * (lane & 3) + e) >> (lane / 4);
#pragma unroll
                  for (int j = 0; j < 2; j++) {
                    bits[0] |= ((v >> (8 * j)) & 1u) << (4 * k + 2 * j + e);
                    bits[1] |= ((v >> (16 + 8 * j)) & 1u) << (4 * k + 2 * j + e);
                  }
                }
#pragma unroll 1
              for (int hf = 0; hf < 2; hf++) {
                const uint32_t ta = ts + ((uint32_t)(16 * hf) << 16) + 64 * ch;
                const uint32_t bh = hf ? bits[1] : bits[0];
                uint32_t z[32];
                tmem_frag8(ta, z);
                tmem_wait(z);
#pragma unroll
                for (int e = 0; e < 32; e++)
                  if (!((bh >> e) & 1u)) z[e] = __float_as_uint(hidden);
                tmem_put(ta, z);
              }
            }
          }
          if (sm.special[team].large) {  // (team-uniform: this job raises the references first)
            if (wt < cols) nb[wt] = -kUnset;
            named_sync(bar, 128);
          }
        }
        for (;;) {
          // the job's weights on the references at hand, their sums apart from
          // the run's until the vote; 64 rows by 16 keys of the warp at a time,
          // the next ones on their way from tensor memory meanwhile
          float ls[32], top = -INFINITY;
          if (ok) {
            uint32_t z[2][32];
            tmem_frag8(ts, z[0]);
            // P of the team's last job has been read, O holds its product
            if (sc > 0)
              ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.pvdone + team), (sc - 1) & 1,
                                                             &sm.failed));
#pragma unroll
            for (int ch = 0; ch < 2; ch++) {
              float nbr[16];  // −reference of rows 64·ch + 8k + 2·(t%4) + {0, 1}
#pragma unroll
              for (int k = 0; k < 8; k++) {
                const float2 n2 =
                    *reinterpret_cast<const float2 *>(nb + 64 * ch + 8 * k + 2 * (lane & 3));
                nbr[2 * k] = n2.x;
                nbr[2 * k + 1] = n2.y;
              }
#pragma unroll
              for (int hf = 0; hf < 2; hf++) {
                const int w = 2 * ch + hf;
                tmem_wait(z[w & 1]);
                if (w < 3)
                  tmem_frag8(ts + ((uint32_t)(16 * ((w + 1) & 1)) << 16) + 64 * ((w + 1) >> 1),
                               z[(w + 1) & 1]);
                float x[32];
#pragma unroll
                for (int e = 0; e < 32; e++)
                  x[e] = fmaf(__uint_as_float(z[w & 1][e]), zs, nbr[(e >> 2) * 2 + (e & 1)]);
#pragma unroll
                for (int e = 0; e < 32; e += 2) top = max3(top, x[e], x[e + 1]);
#pragma unroll
                for (int e = 0; e < 32; e++) x[e] = ex2(x[e]);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                  const float s0 = x[4 * k] + x[4 * k + 2], s1 = x[4 * k + 1] + x[4 * k + 3];
                  ls[16 * ch + 2 * k] = hf ? ls[16 * ch + 2 * k] + s0 : s0;
                  ls[16 * ch + 2 * k + 1] = hf ? ls[16 * ch + 2 * k + 1] + s1 : s1;
                }
                const uint32_t pa = pst + ch * 8192 + (((mchunk + hf * 2) ^ (mrow & 7)) << 4);
#pragma unroll
                for (int k = 0; k < 8; k += 2)
                  stsm4t(pa + k * 1024, pack_bf16x2(x[4 * k], x[4 * k + 1]),
                         pack_bf16x2(x[4 * k + 2], x[4 * k + 3]),
                         pack_bf16x2(x[4 * k + 4], x[4 * k + 5]),
                         pack_bf16x2(x[4 * k + 6], x[4 * k + 7]));
              }
            }
          }
          // the vote also keeps the team's warps within one job of each other
          const bool raise = named_sync_or(bar, 128, !ok || top > kExceed);
          if (!raise) {
#pragma unroll
            for (int e = 0; e < 32; e++) l[e] += ls[e];
            break;
          }
          ok = named_sync_and(bar, 128, ok);
          if (!ok) break;
#pragma unroll 1
          for (int ch = 0; ch < 2; ch++) {
            float cm[16];
#pragma unroll
            for (int e = 0; e < 16; e++) cm[e] = -INFINITY;
#pragma unroll 1
            for (int hf = 0; hf < 2; hf++) {
              uint32_t z[32];
              tmem_frag8(ts + ((uint32_t)(16 * hf) << 16) + 64 * ch, z);
              tmem_wait(z);
#pragma unroll
              for (int e = 0; e < 32; e++)
                cm[(e >> 2) * 2 + (e & 1)] =
                    fmaxf(cm[(e >> 2) * 2 + (e & 1)], __fmul_rn(__uint_as_float(z[e]), zs));
            }
#pragma unroll
            for (int e = 0; e < 16; e++) {
#pragma unroll
              for (int o = 4; o < 32; o <<= 1)
                cm[e] = fmaxf(cm[e], __shfl_xor_sync(0xFFFFFFFFu, cm[e], o));
              if (lane < 4) scr[quarter * 128 + 64 * ch + (e >> 1) * 8 + 2 * lane + (e & 1)] = cm[e];
            }
          }
          named_sync(bar, 128);
          bool large = false;
          {
            float f = 1.f;
            if (wt < cols) {
              const float was = sm.special[team].large ? large_ref[0] : -nb[wt];
              const float m =
                  fmaxf(fmaxf(scr[wt], scr[128 + wt]), fmaxf(scr[256 + wt], scr[384 + wt]));
              const float now = fmaxf(was, m);
              f = ex2(was - now);
              nb[wt] = -now;
              large_ref[0] = now;
              large = m > -INFINITY && fabsf(now) >= kRoundFrom;
            }
            scr[512 + wt] = f;
          }
          large = named_sync_or(bar, 128, large || sm.special[team].large);
          const float *fac = scr + 512;
#pragma unroll
          for (int e = 0; e < 32; e++) {
            const int x = 8 * (e >> 1) + 2 * (lane & 3) + (e & 1);
            if (x < cols) l[e] *= fac[x];
          }
          if (!fresh) {  // O's lanes are the team's rows
            const float f = fac[quarter * 32 + lane];
            tc_fence_after();  // (after the wait for pvdone: the product that wrote O)
#pragma unroll 1
            for (int cc = 0; cc < D; cc += 16) {
              float v[16];
              tmem_ld16(to + cc, v);
#pragma unroll
              for (int e = 0; e < 16; e++) v[e] *= f;
              tmem_st16(to + cc, v);
            }
          }
          if (large) {  // Sᵀ ← (fl(Sᵀ·zscale) − reference) / zscale; the loop's references are 0
#pragma unroll 1
            for (int w = 0; w < 4; w++) {
              const uint32_t ta = ts + ((uint32_t)(16 * (w & 1)) << 16) + 64 * (w >> 1);
              uint32_t z[32];
              tmem_frag8(ta, z);
              tmem_wait(z);
#pragma unroll
              for (int e = 0; e < 32; e++)
                z[e] = __float_as_uint(
                    __fadd_rn(__fmul_rn(__uint_as_float(z[e]), zs),
                              nb[64 * (w >> 1) + 8 * (e >> 2) + 2 * (lane & 3) + (e & 1)]) / zs);
              tmem_put(ta, z);
            }
            named_sync(bar, 128);
            if (wt < cols) nb[wt] = 0.f;
            sm.special[team].large = 1;
          }
          named_sync(bar, 128);  // the factors are read before P replaces them
        }
        if (!ok) break;
        tc_fence_before();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(sm.sfree + team));
          mbar_arrive(smem_u32(sm.pready + team));
        }
        fresh = false;
      }
      // ---- the run's result: sums over the key lanes, then O
      if (ok && !fresh)
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.pvdone + team), (sc - 1) & 1,
                                                       &sm.failed));
      ok = named_sync_and(bar, 128, ok);
      tc_fence_after();
      // (max, sum) per row in the second half of P, free like the first (its last
      // product is done)
      float2 *ml = reinterpret_cast<float2 *>(p_team + kTtP / 2);
      if (ok) {
#pragma unroll
        for (int e = 0; e < 32; e++) {
          float x = l[e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
          if (lane < 4) scr[quarter * 128 + 8 * (e >> 1) + 2 * lane + (e & 1)] = x;
        }
      }
      named_sync(bar, 128);
      if (ok) {
        const float sum = (scr[wt] + scr[128 + wt]) + (scr[256 + wt] + scr[384 + wt]);
        const bool any = wt < cols && (sum > 0.f || sum != sum);
        const float m = sm.special[team].large ? large_ref[0] : -nb[wt];
        ml[wt] = make_float2(any ? m : -INFINITY, any ? sum : 0.f);
      }
      ok = named_sync_and(7, kTtSoft * 32, ok);
      if (!ok) break;
      // every warp: its quarter's row of each team, half of the columns
      const int lr = quarter * 32 + lane;
      const float2 *mls = reinterpret_cast<const float2 *>(base + kTtHead + kTtP / 2) + lr;
      const float2 ml0 = mls[0], ml1 = mls[kTtP / 8];
      named_sync(7, kTtSoft * 32);
      const bool whole = t0 == 0 && t1 == pos.n_kt;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (pos.g != pos.run0);
      const int h = pos.h();
      const bool odd = sm.odd != 0;
      constexpr int W = D / 2;  // columns per warp
      const int d0 = team * W;
#pragma unroll 1
      for (int part = 0; part < (halves ? 2 : 1); part++) {
        const int row = part * 128 + lr;
        if (part * 128 + quarter * 32 >= n_rows) break;  // warp-uniform
        // one team's rows, or both teams' shares of the same rows
        const float2 mlp = part ? ml1 : ml0;
        const float m = halves ? mlp.x : fmaxf(ml0.x, ml1.x);
        const float m_use = m == -INFINITY ? 0.f : m;
        float f0, f1 = 0.f, sum;
        if (halves) {
          f0 = 1.f;
          sum = mlp.y;
        } else {
          f0 = ex2(ml0.x - m_use);
          f1 = ex2(ml1.x - m_use);
          sum = fmaf(ml0.y, f0, ml1.y * f1);
        }
        // (a team that saw nothing of the row may hold anything; one whose weights
        // are all below fp32 still holds NaN where a value is not finite)
        const bool s0 = halves ? m > -INFINITY : ml0.x > -INFINITY, s1 = !halves && ml1.x > -INFINITY;
        const float inv = whole ? (m == -INFINITY ? 0.f : 1.f / sum) : 1.f;
        const bool two = !halves && t1 - t0 > 1;
        const int x = pos.rt() * a.rstep + row, i = x / a.G;
        const int64_t qr = (int64_t)(pos.q0 + i) * a.Hq + h * a.G + x % a.G;
        const bool mine = row < n_rows;
#pragma unroll 1
        for (int cc = 0; cc < W; cc += 16) {
          float v[16], u[16];
          tmem_ld16(tmem + 256 + (halves ? part * 128 : 0) + lanes + d0 + cc, v);
          if (two) tmem_ld16(tmem + 256 + 128 + lanes + d0 + cc, u);
#pragma unroll
          for (int e = 0; e < 16; e++) {
            v[e] = s0 ? v[e] * f0 : 0.f;
            if (two && s1) v[e] = fmaf(u[e], f1, v[e]);
          }
          if (odd && mine) {  // infinities and NaN of the nodes this run covered that the row sees
            const int j1 = min(pos.T, t1 * kTtKeys - pos.c);
#pragma unroll 1
            for (int jn = max(0, t0 * kTtKeys - pos.c); jn < j1; jn++) {
              const bool see_n = a.mask ? (a.mask[(int64_t)(pos.q0 + i) * a.mask_words + (jn >> 5)] >> (jn & 31)) & 1u
                                        : jn <= i;
              const int pn = pos.c + jn, pg = page_of(pn, a.bs_inv);
              const int32_t bn = bt[pg];
              if (!see_n || bn < 0 || bn >= n_blocks) continue;
              const uint16_t *vr =
                  a.vpool + (((int64_t)bn * a.BS + pn - pg * a.BS) * a.H + h) * D + d0 + cc;
#pragma unroll
              for (int e = 0; e < 16; e++) {
                const float vn = bf16_lo(vr[e]);
                if (!(fabsf(vn) < INFINITY)) v[e] += vn;
              }
            }
          }
          if (!mine) continue;
          if (whole) {
            uint4 o[2];
            uint32_t *ow = reinterpret_cast<uint32_t *>(o);
#pragma unroll
            for (int e = 0; e < 8; e++) ow[e] = pack_bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + qr * D + d0 + cc);
            dst[0] = o[0];
            dst[1] = o[1];
          } else {
            float4 *dst = reinterpret_cast<float4 *>(a.part_o + (slot * a.rows + row) * D + d0 + cc);
#pragma unroll
            for (int e = 0; e < 4; e++)
              dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        }
        if (mine && d0 == 0) {
          if (whole) a.lse[qr] = m == -INFINITY ? -INFINITY : (m + log2f(sum)) * kLn2;
          else a.part_ml[slot * a.rows + row] = make_float2(m, sum);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.ofree));
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
    for (int i = 0; i < 2 * kTtSlots; i++) {
      mbar_drain(smem_u32(sm.full[0] + i), 0);
      mbar_drain(smem_u32(sm.full[0] + i), 1);
    }
    mbar_drain(smem_u32(&sm.qfull), 0);
    mbar_drain(smem_u32(&sm.qfull), 1);
    for (int i = 0; i < 2; i++) {
      mbar_drain(smem_u32(sm.sfull + i), 0);
      mbar_drain(smem_u32(sm.sfull + i), 1);
      mbar_drain(smem_u32(sm.pvdone + i), 0);
      mbar_drain(smem_u32(sm.pvdone + i), 1);
    }
  }
  __syncthreads();
  if (warp == kTtSoft + 4) {
    tc_fence_after();
    free_tmem_cols(tmem, 512);
  }
}

// Rows up to which the narrow instruction is used.  Both sides, 64 requests of
// 8K: 4 rows 250 us here and 294 on the tensor cores, 16 rows 256 and 298, 32
// rows 287 and 303; 1K of one request, 16 rows 11 and 20; 128K, 32 rows 108 and
// 105.
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

template <int D>
cudaError_t launch_tc(const TreeArgs &a, cudaStream_t s) {
  constexpr size_t kSmemMax = 232448;
  TreeTc p;
  p.NS = 1024 + TreeTcSmem(D, a.rows, kTtSlots).bytes <= kSmemMax ? kTtSlots : 3;
  CUtensorMap tm_k{}, tm_v{}, tm_q{};
  p.box = a.BS % 32 == 0 ? 32 : a.BS % 16 == 0 ? 16 : a.BS % 8 == 0 ? 8 : 0;
  if (p.box && !(pool_map(&tm_k, a.kpool, a.n_slots, a.H, D, p.box) &&
                 pool_map(&tm_v, a.vpool, a.n_slots, a.H, D, p.box)))
    return cudaErrorUnknown;
  p.q_nodes = a.rstep / a.G;
  if (!q_map(&tm_q, a.q, a.n_q, a.Hq, D, a.G, p.q_nodes)) return cudaErrorUnknown;
  p.idesc_s = make_idesc(128, 0);
  p.idesc_o = make_idesc(128, D) | (1u << 16);  // B (V) MN-major
  const size_t smem = 1024 + TreeTcSmem(D, a.rows, p.NS).bytes;
  // (the limit is the process's: the largest, so that no thread's call lowers it
  // under another's launch)
  cudaError_t e = cudaFuncSetAttribute(
      k_tree_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
  if (e != cudaSuccess) return e;
  static std::atomic<int> regs{0};  // a thread's registers at launch
  if (!regs.load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa{};
    if ((e = cudaFuncGetAttributes(&fa, k_tree_tc<D>)) != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  // setmaxnreg.inc draws on what the block was launched with
  if (regs.load(std::memory_order_relaxed) * kTtThreads < 256 * (kTtMore + kTtLess))
    return cudaErrorLaunchOutOfResources;
  k_tree_tc<D><<<a.n_cta, kTtThreads, smem, s>>>(tm_k, tm_v, tm_q, a, p);
  return cudaGetLastError();
}

// CTAs of the cluster that shares a unit, 0: the tiles are dealt out and joined.
// In tiles that a CTA takes one after another.  Dealt out: an even share, which at D
// 64 and one row tile takes 1.2 times as long, and about 17 (the join's launch and
// dependent loads, a second start).  Clusters: a share for every wave of CTAs, of
// which the last is charged by what it holds and 0.6 of the rest (its CTAs begin as
// the others end), 5 to start each wave after the first, and 3.5; 16 CTAs leave some
// SMs empty.  Both sides measured at 1474 sizes, 1 to 64 requests of 300 to 16K, 2 to
// 16 heads, 4 to 32 rows: the form chosen takes 0.7 % longer than the best one in the
// mean, and over 5 % longer at 67 (the most with 32 rows of D 64).
// One token, 8 KV heads, 1 request: 4K 10.8 us by clusters of 16 and 12.6 dealt out,
// 16K 21.7 and 17.4.  12 rows, 16 heads of D 64: 24 requests of 6K 107 us by clusters
// of two and 115, of 8K 130 and 140, 48 of 4K 133 by single CTAs and 144.
int tree_cluster(const TreeArgs &a, int D) {
  const double units = (double)a.n_req * a.H, sms = device_sm_count();
  const double kt = ceil((double)a.max_blocks * a.BS / a.tile);
  int best = 0;
  double least = (D == 64 && a.rows == 16 ? 1.2 : 1) * units * kt / (2 * sms) + 17;
  for (int S = 1; S <= 16 && S <= kt; S *= 2) {
    // (two CTAs per SM; a GPC's 16 to 20 SMs hold fewer large clusters)
    const double room = S == 16 ? 0.85 * sms : S == 8 ? 1.69 * sms : S == 4 ? 1.9 * sms : 2 * sms;
    const double full = units * S / room, waves = ceil(full);
    const double share = waves > 1 ? full + 0.6 * (waves - full) : 1;
    const double cost = share * ceil(kt / S) * (S == 16 ? 1.25 : 1) + 5 * (waves - 1) + 3.5;
    if (cost < least) {
      least = cost;
      best = S;
    }
  }
  return units * best <= INT32_MAX ? best : 0;
}

template <int D, int MT>
cudaError_t launch_rows(const TreeArgs &a, int cluster, cudaStream_t s) {
  constexpr int smem = RowSmem<D, MT>::kBytes;
  auto *kern = cluster ? k_tree_rows<D, MT, true> : k_tree_rows<D, MT, false>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && cluster > 8)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster ? (unsigned)(a.n_req * a.H * cluster) : (unsigned)a.n_cta);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
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
  a.bs_inv = page_inverse(BS);
  a.zscale = scale != 0.f ? scale * kLog2e : 1e-30f;  // (so that −inf stays −inf when scaled)
  int max_rt;
  tree_plan(n_req, max_blocks, max_tree, H, Hq, D, BS, a.rows, a.rstep, a.tile, a.n_cta, max_rt);
  a.part_o = reinterpret_cast<float *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)2 * a.n_cta * a.rows * D);
  cudaError_t e;
  const int cluster = max_tree * a.G > kRowsMax ? 0 : tree_cluster(a, D);
  if (max_tree * a.G > kRowsMax)
    e = D == 128 ? launch_tc<128>(a, s) : launch_tc<64>(a, s);
  else
    e = D == 128 ? (a.rows == 16 ? launch_rows<128, 1>(a, cluster, s) : launch_rows<128, 2>(a, cluster, s))
                 : (a.rows == 16 ? launch_rows<64, 1>(a, cluster, s) : launch_rows<64, 2>(a, cluster, s));
  if (e != cudaSuccess || cluster) return e;
  return launch_join(a, D, max_rt, s);
}

}  // namespace kvc
