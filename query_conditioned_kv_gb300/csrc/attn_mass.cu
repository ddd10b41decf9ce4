// attn_mass.cu — accumulated attention weight per (layer, request, KV head,
// cached position): the rows' softmax weights, recovered from attention's
// LSE, added up over the rows and the heads of the group,
//   mass[p] ← (p < n_mass ? decay·mass[p] : 0)
//             + Σ_{rows i, p < vis_i} Σ_g exp(scale·q_{i,g}·k_p − lse_{i,g})
// In base 2: 2^(z·scale·log2e − lse·log2e), one FMA and one ex2 per weight.
//
// Orientation.  Keys are the M dimension of the product, rows (row, head of
// the group) the N dimension: each thread then holds weights of its own keys
// and adds them up in registers, so the sum over rows costs no exchange
// beyond one step across four lanes, and every position is owned by one
// warp: no atomics, no partial sums in memory.
//
// k_mass_rows (few rows): bound by the stream of K, 2·D bytes per key.  All
// key tiles of all (layer, request, KV head) units, in order, are dealt out
// in equal contiguous runs to the CTAs; each of a CTA's four warps streams
// its 16 (D 128) or 32 (D 64) keys of a tile through a private cp.async ring
// (4 stages of 4 KB).  mma.sync m16n8k16, fp32 accumulators.
#include <math.h>

#include <algorithm>

#include "kvc_internal.cuh"
#include "mma_ptx.cuh"
#include "tc_ptx.cuh"

namespace kvc {
namespace {

using namespace tc;

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

// Request r's sizes; false when they are out of range.
__device__ __forceinline__ bool mass_request(const MassArgs &a, int r, int &seq, int &r0, int &n) {
  seq = a.seqused[r];
  r0 = a.row_off[r];
  const int64_t m = (int64_t)a.row_off[r + 1] - r0;
  n = (int)m;
  return seq >= 0 && seq <= a.cap && r0 >= 0 && m >= 0 && m <= a.max_rows && r0 + m <= a.n_rows;
}

// ---------------------------------------------------------------- few rows

constexpr int kMrWarps = 4;
constexpr int kMrThreads = kMrWarps * 32;
constexpr int kMrStages = 4;
constexpr int kMrStage = 4096;  // bytes of one warp's stage

template <int D, int NT>  // NT 8-row tiles of query rows
struct MassRowSmem {
  static constexpr int kRing = kMrWarps * kMrStages * kMrStage;
  static constexpr int kQ = kRing;
  static constexpr int kLse = kQ + NT * 8 * D * 2;  // lse·log2e per row
  static constexpr int kVis = kLse + NT * 8 * 4;    // positions each row sees
  static constexpr int kMisc = kVis + NT * 8 * 4;   // scan scratch [66] int64
  static constexpr int kValid = kMisc + 66 * 8;
  static constexpr int kBytes = kValid + kMrWarps * kMrStages * 4;
};

// Key tiles of all requests (per layer and head), by the whole CTA.
__device__ __forceinline__ int mass_tiles(const MassArgs &a, int r, int tile) {
  int seq, r0, n;
  return mass_request(a, r, seq, r0, n) ? (seq + tile - 1) / tile : 0;
}

template <int D, int NT>
__global__ void __launch_bounds__(kMrThreads)
k_mass_rows(MassArgs a, int n_cta_max) {
  using S = MassRowSmem<D, NT>;
  constexpr int KT = 2048 / D, KS = D / 16, CH = D / 8, MT = KT / 16;
  constexpr int kTile = kMrWarps * KT;
  constexpr bool kQRegs = NT <= 2;  // two row tiles stay in registers
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t *sh = reinterpret_cast<int64_t *>(sm + S::kMisc);
  const uint32_t ring = smem_u32(sm) + warp * kMrStages * kMrStage;
  uint32_t *valid_s = reinterpret_cast<uint32_t *>(sm + S::kValid) + warp * kMrStages;
  float *lse_s = reinterpret_cast<float *>(sm + S::kLse);
  int *vis_s = reinterpret_cast<int *>(sm + S::kVis);
  const uint32_t qbase = smem_u32(sm + S::kQ);

  // tiles of all requests (one layer and head)
  int64_t per = 0;
  for (int r = tid; r < a.n_req; r += kMrThreads) {
    per += mass_tiles(a, r, kTile);
    int seq, r0, n;
    if (blockIdx.x == 0 && !mass_request(a, r, seq, r0, n)) record_error(a.status, KVC_ERR_BOUNDS);
  }
  per = block_sum(per, sh);
  const int64_t total = per * a.L * a.H;
  const int n_cta = (int)min((int64_t)n_cta_max, total);
  if ((int)blockIdx.x >= n_cta) return;
  const int64_t run0 = total * blockIdx.x / n_cta, run1 = total * (blockIdx.x + 1) / n_cta;

  // run0 → (layer, request, head, tile): order l, r, h, tile
  int64_t l = run0 / (per * a.H), in_layer = run0 % (per * a.H), before;
  int r;
  block_find(
      a.n_req, in_layer, sh, [&](int x) { return (int64_t)a.H * mass_tiles(a, x, kTile); }, r, before);
  int n_kt = mass_tiles(a, r, kTile);
  int h = (int)((in_layer - before) / n_kt), t0 = (int)((in_layer - before) % n_kt);
  const int64_t n_blocks = a.n_slots / a.BS;

  for (int64_t g = run0; g < run1;) {
    int seq, r0, n;
    mass_request(a, r, seq, r0, n);
    const int t1 = (int)min((int64_t)n_kt, t0 + (run1 - g));
    const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
    const uint16_t *kl = a.kpool + (l * a.n_slots * a.H + h) * D;

    auto issue = [&](int t, int st) {
      const int p0 = t * kTile + warp * KT;
      int32_t slot = -1;
      if (lane < KT && p0 + lane < seq) {
        const int p = p0 + lane;
        const int32_t b = bt[p / a.BS];
        if (b >= 0 && b < n_blocks) slot = b * a.BS + p % a.BS;
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
        cp_async16(ring + st * kMrStage + swz<D>(row, col),
                   kl + (int64_t)max(sl, 0) * a.H * D + col * 8, sl >= 0);
      }
    };
#pragma unroll
    for (int s = 0; s < kMrStages - 1; s++) {
      if (t0 + s < t1) issue(t0 + s, s);
      cp_commit();
    }
    // this unit's query rows, their LSE and limits
    const int n_rows = n * a.G;
    for (int e = tid; e < NT * 8 * CH; e += kMrThreads) {
      const int row = e / CH, col = e % CH;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < n_rows) {
        const int i = r0 + row / a.G, x = a.row_idx ? a.row_idx[i] : i;
        if (x >= 0 && x < a.n_q)
          v = *reinterpret_cast<const uint4 *>(
              a.q + ((l * a.n_q + x) * a.Hq + h * a.G + row % a.G) * D + col * 8);
      }
      *reinterpret_cast<uint4 *>(sm + S::kQ + swz<D>(row, col)) = v;
    }
    // Rows that add nothing get lse = +inf, so their weight is 0 wherever K is
    // finite; `lo`, the least limit of the others, tells the tiles that every
    // one of them sees (there a NaN key is a NaN result in any case).
    int lo = seq + 1;
    for (int row = tid; row < NT * 8; row += kMrThreads) {
      float ls = INFINITY;
      int vis = 0;
      if (row < n_rows) {
        const int i = r0 + row / a.G, x = a.row_idx ? a.row_idx[i] : i;
        vis = min(a.row_vis[i], seq);
        if (vis > 0 && x >= 0 && x < a.n_q) {
          ls = a.lse[(l * a.n_q + x) * a.Hq + h * a.G + row % a.G] * kLog2e;
          if (ls == -INFINITY) ls = INFINITY;
          else lo = min(lo, vis);
        } else if (vis > 0) {
          record_error(a.status, KVC_ERR_BOUNDS);
        }
      }
      lse_s[row] = ls;
      vis_s[row] = ls == INFINITY ? 0 : vis;
    }
    lo = -(int)block_max(-lo, sh);  // (its barriers publish q, lse and limits)
    if (lo > seq) lo = 0;           // no row adds anything

    uint32_t qf[kQRegs ? KS : 1][NT][2];
    if (kQRegs)
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        uint32_t b[4];
        ldsm4(qbase + swz<D>(NT == 1 ? (lane & 7) : (lane & 7) + ((lane >> 4) << 3),
                             2 * ks + ((lane >> 3) & 1)), b);
#pragma unroll
        for (int nt = 0; nt < NT && nt < 2; nt++) {
          qf[kQRegs ? ks : 0][nt][0] = b[2 * nt];
          qf[kQRegs ? ks : 0][nt][1] = b[2 * nt + 1];
        }
      }
    float *out = a.mass + (((int64_t)l * a.n_req + r) * a.H + h) * a.cap;
    const int n_old = a.n_mass[r];

    int st = 0;
    for (int t = t0; t < t1; t++) {
      cp_wait<kMrStages - 2>();
      __syncwarp();
      const int nx = t + kMrStages - 1;
      if (nx < t1) issue(nx, (st + kMrStages - 1) % kMrStages);
      cp_commit();
      const uint32_t kb = ring + st * kMrStage;
      const int p0 = t * kTile + warp * KT;
      const uint32_t okb = valid_s[st];
      // the weight already there, fetched while the product runs
      const int pw = p0 + lane;
      const bool mine = lane < KT && pw < seq;
      const float old = mine && pw < n_old ? out[pw] : 0.f;
      float c[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++) c[mt][nt][0] = c[mt][nt][1] = c[mt][nt][2] = c[mt][nt][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        uint32_t ka[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
          ldsm4(kb + swz<D>(mt * 16 + (lane & 15), 2 * ks + (lane >> 4)), ka[mt]);
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
          uint32_t b[4];
          if (kQRegs) {
            b[0] = qf[kQRegs ? ks : 0][0][0];
            b[1] = qf[kQRegs ? ks : 0][0][1];
            if (NT > 1) {
              b[2] = qf[kQRegs ? ks : 0][NT > 1 ? 1 : 0][0];
              b[3] = qf[kQRegs ? ks : 0][NT > 1 ? 1 : 0][1];
            }
          } else {
            ldsm4(qbase + swz<D>(nt * 8 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), b);
          }
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            mma16816(c[mt][nt], ka[mt], b[0], b[1]);
            if (nt + 1 < NT) mma16816(c[mt][nt + 1 < NT ? nt + 1 : nt], ka[mt], b[2], b[3]);
          }
        }
      }
      // keys lane/4 and lane/4 + 8 of each m tile; rows 2·(lane%4) + {0, 1} of each n tile
      const bool masked = p0 + KT > lo;  // some row stops inside or before the tile
      float sum[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; mt++) sum[mt][0] = sum[mt][1] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        const float2 ls = *reinterpret_cast<const float2 *>(lse_s + nt * 8 + 2 * (lane & 3));
        const int2 vs = *reinterpret_cast<const int2 *>(vis_s + nt * 8 + 2 * (lane & 3));
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
            float w0 = ex2(fmaf(c[mt][nt][2 * hf], a.zscale, -ls.x));
            float w1 = ex2(fmaf(c[mt][nt][2 * hf + 1], a.zscale, -ls.y));
            if (masked) {
              const int p = p0 + mt * 16 + hf * 8 + lane / 4;
              w0 = p < vs.x ? w0 : 0.f;
              w1 = p < vs.y ? w1 : 0.f;
            }
            sum[mt][hf] += w0 + w1;
          }
      }
      float res = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
          float x = sum[mt][hf];
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
          // key mt·16 + hf·8 + k is in lanes 4k … 4k + 3: hand it to lane of that key
          x = __shfl_sync(0xFFFFFFFFu, x, (lane & 7) << 2);
          if ((lane >> 3) == mt * 2 + hf) res = x;
        }
      if (mine) out[pw] = fmaf(a.decay, old, (okb >> lane) & 1u ? res : 0.f);
      st = (st + 1) % kMrStages;
    }
    cp_wait<0>();
    g += t1 - t0;
    t0 = 0;
    if (g < run1 && t1 == n_kt && ++h == a.H) {
      h = 0;
      do {
        if (++r == a.n_req) {
          r = 0;
          l++;
        }
        n_kt = mass_tiles(a, r, kTile);
      } while (n_kt == 0);  // g < run1 ≤ total: a later request holds tile g
    }
    __syncthreads();
  }
}

template <int D, int NT>
cudaError_t launch_rows(const MassArgs &a, cudaStream_t s) {
  constexpr int smem = MassRowSmem<D, NT>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(k_mass_rows<D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int per_sm = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_mass_rows<D, NT>, kMrThreads, smem);
  if (e != cudaSuccess) return e;
  constexpr int tile = kMrWarps * 2048 / D;
  const int64_t most = (int64_t)a.L * a.n_req * a.H * ((a.cap + tile - 1) / tile);
  const int n_cta = (int)std::min<int64_t>((int64_t)std::min(per_sm, 3) * device_sm_count(), most);
  k_mass_rows<D, NT><<<n_cta, kMrThreads, smem, s>>>(a, n_cta);
  return cudaGetLastError();
}

// --------------------------------------------------------------- many rows

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
  const int64_t R = (int64_t)max_rows * a.G;
  if (R <= 64) {
    if (D == 128)
      return R <= 8    ? launch_rows<128, 1>(a, s)
             : R <= 16 ? launch_rows<128, 2>(a, s)
             : R <= 32 ? launch_rows<128, 4>(a, s)
                       : launch_rows<128, 8>(a, s);
    return R <= 8    ? launch_rows<64, 1>(a, s)
           : R <= 16 ? launch_rows<64, 2>(a, s)
           : R <= 32 ? launch_rows<64, 4>(a, s)
                     : launch_rows<64, 8>(a, s);
  }
  const int segs = L * n_req * H, y = segs < 32768 ? segs : 32768;
  const dim3 grid((a.cap + 7) / 8, y, (segs + y - 1) / y);
  if (D == 128) k_attn_mass<128><<<grid, 256, 0, s>>>(a);
  else k_attn_mass<64><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
