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
#include <limits.h>
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
  uint32_t bs_inv;  // page_inverse(BS)
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
constexpr int kMrMaxRows = 64;  // widest row set (rows · G) of this path
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
        cp_async16(ring + st * kMrStage + swz<D>(row, col),
                   kl + (int64_t)max(sl, 0) * a.H * D + col * 8, sl >= 0);
      }
    };
#pragma unroll
    for (int s = 0; s < kMrStages - 1; s++) {
      if (t0 + s < t1) issue(t0 + s, s);
      cp_commit();
    }
    // this unit's rows: LSE and limits, then the queries.  A row that adds
    // nothing (past the request's rows, no limit, LSE ±inf) gets lse = +inf and
    // q = 0, so its weight is 0 wherever K is finite; `lo`, the least limit of
    // the others, tells the tiles that every one of them sees (there a NaN key
    // is a NaN result in any case).
    const int n_rows = n * a.G;
    int lo = seq + 1;
    for (int row = tid; row < NT * 8; row += kMrThreads) {
      float ls = INFINITY;
      int vis = 0;
      if (row < n_rows) {
        const int i = r0 + row / a.G, x = a.row_idx ? a.row_idx[i] : i;
        vis = min(a.row_vis[i], seq);
        if (vis > 0 && x >= 0 && x < a.n_q) {
          ls = a.lse[(l * a.n_q + x) * a.Hq + h * a.G + row % a.G] * kLog2e;
          if (fabsf(ls) == INFINITY) ls = INFINITY;
          else lo = min(lo, vis);
        } else if (vis > 0) {
          record_error(a.status, KVC_ERR_BOUNDS);
        }
      }
      lse_s[row] = ls;
      vis_s[row] = ls == INFINITY ? 0 : vis;
    }
    lo = -(int)block_max(-lo, sh);  // (its barriers publish lse and limits)
    if (lo > seq) lo = 0;           // no row adds anything
    for (int e = tid; e < NT * 8 * CH; e += kMrThreads) {
      const int row = e / CH, col = e % CH;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (lse_s[row] != INFINITY) {
        const int i = r0 + row / a.G, x = a.row_idx ? a.row_idx[i] : i;
        v = *reinterpret_cast<const uint4 *>(
            a.q + ((l * a.n_q + x) * a.Hq + h * a.G + row % a.G) * D + col * 8);
      }
      *reinterpret_cast<uint4 *>(sm + S::kQ + swz<D>(row, col)) = v;
    }
    __syncthreads();
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
//
// tcgen05: D[key][row] = K tile (M 128 keys, A) × row tile (N rows, B), fp32 in
// tensor memory.  Warps 0–7: two epilogue warpgroups, taking the key tiles in
// turn; 8–11: producers; 12–13: one MMA warp for each epilogue warpgroup (a
// warp's waits run under the other's products).  An epilogue thread owns four
// keys and a quarter of the rows (16x256b fragments): the rows' LSE, stored in
// that order, costs it a quarter of the shared-memory reads that one key a
// thread would, and the sum over rows stays in registers until the group ends.
//
// ONE (all rows of a request in one row tile): the rows stay in shared memory
// while the request's keys stream past; work is dealt out by key tile.
// Otherwise a work item is a group of two key tiles (256 keys, resident) that
// the row tiles stream past (a row tile's 64 KB from L2 feed two products).
// k_mass_plan lists each group's row tiles, those with a row that sees the
// group's first key: under a causal limit the work halves.  All items' row
// tiles, in order, are dealt out in equal contiguous runs to the CTAs; a run
// that holds part of a group writes partial sums, which k_mass_join adds in
// order.

constexpr int kTcEpi = 8;                       // epilogue warps
constexpr int kTcProd = 4;                      // producer warps
constexpr int kTcThreads = (kTcEpi + kTcProd + 2) * 32;
constexpr int kTcKeys = 128;                    // keys of a tile
constexpr int kTcMaxK = 8;                      // K slots, at most
constexpr int kTcQs = 4;                        // slots of 64 columns of a row tile

struct MassTc {
  int n_cta;        // CTAs the work is dealt out to
  int NR;           // rows of a row tile's buffers: 128 or 256
  int tokens;       // rows i (tokens) of a row tile: tokens·G ≤ NR rows
  int k_slots;      // K ring
  int box;          // rows of a TMA box of K (a divisor of the page size), 0: none
  int q_box;        // queries by TMA (no row_idx)
  int max_kg, max_rt;
  uint32_t idesc;
  int64_t *cum;     // [n_req][max_kg + 1]: row tiles before each group (at least one each)
  int2 *span;       // [n_req][max_kg]: first row tile and their number (0: nobody sees the group)
  int *rt_vis;      // [n_req][max_rt]: positions the widest row of the tile sees
  float *part;      // [2·n_cta][256]: partial sums
};

template <bool ONE>
struct TcShape {
  static constexpr int kKG = ONE ? 1 : 2;   // key tiles of a group
  static constexpr int kLs = ONE ? 2 : 4;   // LSE slots
};

// Head of the dynamic shared memory (fixed offsets), then K, q, and the LSE
// slots: −lse·log2e and limits, [slot][NR + 16] in the order of lse_at.
struct TcHead {
  uint64_t kfull[kTcMaxK], kempty[kTcMaxK], qfull[kTcQs], qempty[kTcQs], lfull[4], lempty[4];
  uint64_t tfull[4], tempty[4];
  int64_t scan[66];
  int lo[4][4];  // least limit of the slot's rows, per producer warp
  uint32_t tmem_holder;
  volatile int failed;
};
constexpr uint32_t kTcHead = 1024;
static_assert(sizeof(TcHead) <= kTcHead, "the head's room");

struct TcSmem {
  uint32_t k, q, nlse, vis, bytes;
  __host__ __device__ TcSmem(int D, int NR, int ks, int ls) {
    k = kTcHead;
    q = k + ks * kTcKeys * D * 2;
    nlse = q + kTcQs * NR * 128;
    vis = nlse + ls * (NR + 16) * 4;
    bytes = vis + ls * (NR + 16) * 4;
  }
};

// Place of row r in an LSE slot: the rows 8k + 2q + {0, 1} of an epilogue
// thread (q = lane mod 4) together, quarters four words apart in the banks.
__device__ __forceinline__ int lse_at(int r, int NR) {
  return ((r >> 1) & 3) * (NR / 4 + 4) + (r >> 3) * 2 + (r & 1);
}

// Groups of request r.
__device__ __forceinline__ int tc_groups(const MassArgs &a, int r, int keys) {
  return mass_tiles(a, r, keys);
}

// Where a run stands: group kg of (l, r, h), row tiles [off, cnt) of it left.
template <bool ONE>
struct TcPos {
  int64_t l;
  int r, h, kg, n_kg;
  int rt0, cnt;  // the group's first row tile and their number (0: none)
  int off;       // done by earlier CTAs
  __device__ __forceinline__ void load(const MassArgs &a, const MassTc &p) {
    if (ONE) {
      rt0 = 0;
      cnt = 1;
    } else {
      const int2 s = p.span[(int64_t)r * p.max_kg + kg];
      rt0 = s.x;
      cnt = s.y;
    }
  }
  // the next group (one exists while the run is not over)
  __device__ __forceinline__ void next(const MassArgs &a, const MassTc &p) {
    off = 0;
    if (++kg == n_kg) {
      kg = 0;
      if (++h == a.H) {
        h = 0;
        do {
          if (++r == a.n_req) {
            r = 0;
            l++;
          }
          n_kg = tc_groups(a, r, TcShape<ONE>::kKG * kTcKeys);
        } while (n_kg == 0);
      }
    }
    load(a, p);
  }
};

template <bool ONE>
__device__ __forceinline__ int64_t tc_request_work(const MassArgs &a, const MassTc &p, int r) {
  const int n = tc_groups(a, r, TcShape<ONE>::kKG * kTcKeys);
  return n == 0 ? 0 : ONE ? n : p.cum[(int64_t)r * (p.max_kg + 1) + n];
}

// Position of work item t (by the whole CTA).
template <bool ONE>
__device__ __forceinline__ TcPos<ONE> tc_find(const MassArgs &a, const MassTc &p, int64_t t,
                                              int64_t per, int64_t *sh) {
  TcPos<ONE> x;
  x.l = t / (per * a.H);
  int64_t before;
  const int64_t in_layer = t % (per * a.H);
  block_find(
      a.n_req, in_layer, sh, [&](int r) { return a.H * tc_request_work<ONE>(a, p, r); }, x.r, before);
  const int64_t w = tc_request_work<ONE>(a, p, x.r);
  x.h = (int)((in_layer - before) / w);
  const int64_t in_head = (in_layer - before) % w;
  x.n_kg = tc_groups(a, x.r, TcShape<ONE>::kKG * kTcKeys);
  if (ONE) {
    x.kg = (int)in_head;
    x.off = 0;
  } else {
    const int64_t *cum = p.cum + (int64_t)x.r * (p.max_kg + 1);
    int lo = 0, hi = x.n_kg - 1;  // the last group with cum ≤ in_head
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= in_head) lo = mid;
      else hi = mid - 1;
    }
    x.kg = lo;
    x.off = (int)(in_head - cum[lo]);
  }
  x.load(a, p);
  return x;
}

template <int D, bool ONE>
__global__ void __launch_bounds__(kTcThreads, 1)
k_mass_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
          MassArgs a, MassTc p) {
  constexpr int KG = TcShape<ONE>::kKG, LS = TcShape<ONE>::kLs, QS = kTcQs;
  constexpr int CH = D / 8, KB = D / 64;
  constexpr uint32_t kSlot = kTcKeys * D * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NR = p.NR, KS = p.k_slots, NACC = 512 / NR;
  TcHead &sm = *reinterpret_cast<TcHead *>(base);
  const TcSmem at(D, NR, KS, LS);
  const uint32_t base_u = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    sm.failed = 0;
    for (int i = 0; i < KS; i++) {
      mbar_init(smem_u32(sm.kfull + i), kTcProd * 32);
      mbar_init(smem_u32(sm.kempty + i), 1);
    }
    for (int i = 0; i < QS; i++) {
      mbar_init(smem_u32(sm.qfull + i), kTcProd * 32);
      mbar_init(smem_u32(sm.qempty + i), 2);
    }
    for (int i = 0; i < LS; i++) {
      mbar_init(smem_u32(sm.lfull + i), kTcProd * 32);
      mbar_init(smem_u32(sm.lempty + i), kTcEpi);
    }
    for (int i = 0; i < NACC; i++) {
      mbar_init(smem_u32(sm.tfull + i), 1);
      mbar_init(smem_u32(sm.tempty + i), kTcEpi / 2);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows that no row tile fills stay zero
  if (p.tokens * a.G < NR) {
    for (uint32_t i = tid; i < (uint32_t)kTcQs * NR * 128 / 16; i += kTcThreads)
      *reinterpret_cast<uint4 *>(base + at.q + i * 16) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kTcEpi + kTcProd) alloc_tmem_cols(&sm.tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_holder;

  if (!ONE) asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
  int64_t per = 0;
  for (int r = tid; r < a.n_req; r += kTcThreads) {
    per += tc_request_work<ONE>(a, p, r);
    int seq, r0, n;
    if (ONE && blockIdx.x == 0 && !mass_request(a, r, seq, r0, n))
      record_error(a.status, KVC_ERR_BOUNDS);
  }
  per = block_sum(per, sm.scan);
  const int64_t total = per * a.L * a.H;
  const int n_cta = (int)min((int64_t)p.n_cta, total);
  const bool works = (int)blockIdx.x < n_cta;
  const int64_t run0 = works ? total * blockIdx.x / n_cta : 0;
  const int64_t run1 = works ? total * (blockIdx.x + 1) / n_cta : 0;
  TcPos<ONE> pos{};
  if (works) pos = tc_find<ONE>(a, p, run0, per, sm.scan);
  if (!ONE) asm volatile("griddepcontrol.launch_dependents;");

  bool ok = true;
  if (warp >= kTcEpi && warp < kTcEpi + kTcProd) {
    // ------------------------------------------------------- producers
    // K: 32 keys of a tile a warp, by TMA boxes of whole page rows or row by row
    // with cp.async (bad blocks, the end, page sizes without a box).  Rows: the
    // whole tile in one TMA box, or row by row through row_idx; their LSE and
    // limits through registers, a tile ahead.
    const int pw = warp - kTcEpi;
    const int64_t n_blocks = a.n_slots / a.BS;
    constexpr int RPI = 32 / CH;
    const int col = lane % CH;
    uint32_t kc = 0, qc = 0;      // K tiles and row tiles loaded
    uint32_t pend0 = 0, pend1 = 0;  // stages copied by cp.async and not handed over, oldest first
    int64_t q_unit = -1;
    auto hand = [&](uint32_t bar) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(bar);
    };
    auto flush = [&]() {
      if (!pend0) return;
      cp_wait<0>();
      hand(pend0);
      if (pend1) hand(pend1);
      pend0 = pend1 = 0;
    };
    auto committed = [&](uint32_t bar) {
      cp_commit();
      if (pend1) {
        cp_wait<2>();
        hand(pend0);
        pend0 = pend1;
        pend1 = bar;
      } else if (pend0) {
        pend1 = bar;
      } else {
        pend0 = bar;
      }
    };
    // a full ring is waited for only after everything in flight is handed over
    auto acquire = [&](uint64_t *bar, uint32_t parity) {
      if (mbar_try(smem_u32(bar), parity)) return true;
      flush();
      return mbar_wait_bounded(smem_u32(bar), parity, &sm.failed);
    };
    // this lane's rows of a row tile: lr = 32·pw + 128·u + lane
    const int tok0 = (32 * pw + lane) / a.G, g0 = (32 * pw + lane) % a.G;
    const int tok1 = (32 * pw + lane + 128) / a.G, g1 = (32 * pw + lane + 128) % a.G;
    for (int64_t g = run0; g < run1 && ok;) {
      const int todo = (int)min((int64_t)max(pos.cnt, 1) - pos.off, run1 - g);
      if (pos.cnt > 0) {
        int seq, r0, n;
        mass_request(a, pos.r, seq, r0, n);
        const int32_t *bt = a.block_table + (int64_t)pos.r * a.max_blocks;
        const uint16_t *kl = a.kpool + (pos.l * a.n_slots * a.H + pos.h) * D;
        const float *lse = a.lse + pos.l * a.n_q * a.Hq + pos.h * a.G;
        const int64_t unit = (pos.l * a.n_req + pos.r) * a.H + pos.h;
        const uint32_t uh = uniform32(pos.h);
        auto load_k = [&](int kt) {
          const uint32_t st = kc % KS;
          const int t = pos.kg * KG + kt, pp = t * kTcKeys + pw * 32 + lane;
          int32_t slot = -1;
          if (pp < seq) {
            const int pg = page_of(pp, a.bs_inv);
            const int32_t b = bt[pg];
            if (b >= 0 && b < n_blocks) slot = b * a.BS + pp - pg * a.BS;
            else record_error(a.status, KVC_ERR_BOUNDS);
          }
          if (!(ok = acquire(sm.kempty + st, ((kc / KS) & 1) ^ 1))) return;
          kc++;
          const uint32_t bar = smem_u32(sm.kfull + st);
          const uint32_t slot0 = base_u + at.k + st * kSlot + pw * 32 * 128;
          if (p.box > 0 && __all_sync(0xFFFFFFFFu, slot >= 0)) {
            if (lane == 0) mbar_expect_tx(bar, kSlot / kTcProd);
            else mbar_arrive(bar);
            __syncwarp();
            const uint32_t ubar = uniform32(bar), udst = uniform32(slot0);
            const uint32_t row0 = uniform32((uint32_t)(pos.l * a.n_slots));
            for (int k = 0; k < 32; k += p.box) {
              const uint32_t sl = __shfl_sync(0xFFFFFFFFu, slot, k);
#pragma unroll
              for (int kb = 0; kb < KB; kb++)
                tma_load_3d_if(lane == 0, udst + k * 128 + kb * (kTcKeys * 128), &tm_k, kb * 64, uh,
                               row0 + sl, ubar);
            }
            return;
          }
          const uint32_t dst = slot0 + (col >> 3) * (kTcKeys * 128);
#pragma unroll 4
          for (int i = 0; i < 32 / RPI; i++) {
            const int row = i * RPI + lane / CH;
            const int32_t sl = __shfl_sync(0xFFFFFFFFu, slot, row);
            cp_async16(dst + row * 128 + (((col & 7) ^ (row & 7)) << 4),
                       kl + (int64_t)max(sl, 0) * a.H * D + col * 8, sl >= 0);
          }
          committed(bar);
        };
        // LSE, limit and query row of this lane's rows of row tile rt
        float nl[2];
        int vi[2], qx[2];
        auto fetch = [&](int rt) {
#pragma unroll
          for (int u = 0; u < 2; u++) {
            const int tok = u ? tok1 : tok0, gg = u ? g1 : g0, i = rt * p.tokens + tok;
            nl[u] = -INFINITY;
            vi[u] = 0;
            qx[u] = -1;
            if (tok < p.tokens && i < n && (u == 0 || NR > 128)) {
              const int x = a.row_idx ? a.row_idx[r0 + i] : r0 + i;
              vi[u] = min(a.row_vis[r0 + i], seq);
              if (x >= 0 && x < a.n_q) {
                nl[u] = -lse[(int64_t)x * a.Hq + gg] * kLog2e;
                qx[u] = x;
              } else if (vi[u] > 0) {
                record_error(a.status, KVC_ERR_BOUNDS);
              }
            }
          }
        };
        auto load_q = [&](int rt, bool more) {
          const uint32_t ls = (qc / KB) % LS;
          if (!(ok = acquire(sm.lempty + ls, (((qc / KB) / LS) & 1) ^ 1))) return;
          float *nls = reinterpret_cast<float *>(base + at.nlse) + ls * (NR + 16);
          int *vis = reinterpret_cast<int *>(base + at.vis) + ls * (NR + 16);
          // A row that adds nothing (past the request's rows, no limit, LSE ±inf)
          // has weight 0 by its LSE where its product is finite: its query is
          // zeros, or, where a box brought it along and it may be anything, the
          // tile is masked for every key (lo = 0).
          int lo = INT_MAX;
          int64_t src_row[2];
#pragma unroll
          for (int u = 0; u < 2; u++) {
            src_row[u] = -1;
            if (u == 1 && NR == 128) break;
            const bool on = qx[u] >= 0 && vi[u] > 0 && fabsf(nl[u]) != INFINITY;
            const int r = lse_at(128 * u + 32 * pw + lane, NR);
            nls[r] = on ? nl[u] : -INFINITY;
            vis[r] = on ? vi[u] : 0;
            if (on) lo = min(lo, vi[u]);
            else if (p.q_box && (u ? tok1 : tok0) < p.tokens) lo = 0;
            if (on)
              src_row[u] = (pos.l * a.n_q + qx[u]) * a.Hq + pos.h * a.G + (u ? g1 : g0);
          }
          lo = __reduce_min_sync(0xFFFFFFFFu, lo);
          if (lane == 0) sm.lo[ls][pw] = lo;
          __syncwarp();
          mbar_arrive(smem_u32(sm.lfull + ls));
          if (more) fetch(rt + 1);
          for (int kb = 0; kb < KB; kb++, qc++) {
            const uint32_t st = qc % QS;
            if (!(ok = acquire(sm.qempty + st, ((qc / QS) & 1) ^ 1))) return;
            const uint32_t bar = smem_u32(sm.qfull + st), dst = base_u + at.q + st * (NR * 128);
            if (p.q_box) {
              if (pw == 0 && lane == 0) {
                mbar_expect_tx(bar, p.tokens * a.G * 128);
                tma_load_3d(dst, &tm_q, kb * 64, pos.h * a.G,
                            (int)(pos.l * a.n_q) + r0 + rt * p.tokens, bar);
              } else {
                mbar_arrive(bar);
              }
              continue;
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
              if (u == 1 && NR == 128) break;
#pragma unroll
              for (int i = 0; i < 8; i++) {
                const int rr = i * 4 + lane / 8, c8 = lane % 8;
                const int64_t src = __shfl_sync(0xFFFFFFFFu, src_row[u], rr);
                cp_async16(dst + (128 * u + 32 * pw + rr) * 128 + ((c8 ^ (rr & 7)) << 4),
                           a.q + max(src, (int64_t)0) * D + kb * 64 + c8 * 8, src >= 0);
              }
            }
            committed(bar);
          }
        };
        if (!ONE || unit != q_unit) fetch(pos.rt0 + pos.off);
        load_k(0);
        if (ONE) {
          if (ok && unit != q_unit) {
            load_q(0, false);
            flush();  // (the next stages may all be boxes)
          }
        } else {
          for (int i = 0; i < todo && ok; i++) {
            load_q(pos.rt0 + pos.off + i, i + 1 < todo);
            if (i == 0 && ok) load_k(1);
          }
        }
        q_unit = unit;
      }
      g += todo;
      if (g < run1) pos.next(a, p);
    }
    flush();
    cp_wait<0>();
    if (!ok) sm.failed = 1;
  } else if (warp >= kTcEpi + kTcProd) {
    // ----------------------------------------------------- MMA issuers
    // (the whole warp runs the loop; one lane's products are enabled)
    const int wg = warp - kTcEpi - kTcProd;  // the epilogue warpgroup it works for
    const uint32_t lead = lane == 0;
    uint32_t kc = 0, qc = 0, jc = 0;  // first K tile of the group, q stages, products of both
    int64_t q_unit = -1;
    for (int64_t g = run0; g < run1 && ok;) {
      const int todo = (int)min((int64_t)max(pos.cnt, 1) - pos.off, run1 - g);
      if (pos.cnt > 0) {
        const int64_t unit = (pos.l * a.n_req + pos.r) * a.H + pos.h;
        for (int i = 0; i < todo && ok; i++) {
          if (!ONE || unit != q_unit) {
            if (ONE && qc > 0)
              for (int kb = 0; kb < KB; kb++) mma_commit_if(lead, smem_u32(sm.qempty + (qc - KB + kb) % QS));
            qc += KB;
            // (also for a unit without a tile of this warp's: a barrier's parity
            // tells only two uses apart)
            for (int kb = 0; ONE && kb < KB && ok; kb++)
              ok = mbar_wait_bounded(smem_u32(sm.qfull + (qc - KB + kb) % QS),
                                     ((qc - KB + kb) / QS) & 1, &sm.failed);
            if (!ok) break;
          }
          const uint32_t job = ONE ? jc : jc + wg;
          jc += KG;
          if (ONE && (job & 1) != (uint32_t)wg) continue;
          const uint32_t kx = kc + (ONE ? 0 : wg), kst = kx % KS, acc = job % NACC;
          ok = mbar_wait_bounded(smem_u32(sm.kfull + kst), (kx / KS) & 1, &sm.failed);
          if (ok) ok = mbar_wait_bounded(smem_u32(sm.tempty + acc), ((job / NACC) & 1) ^ 1, &sm.failed);
          const uint64_t kd = uniform64(smem_desc(base_u + at.k + kst * kSlot));
          const uint32_t dst = uniform32(tmem + acc * NR);
#pragma unroll
          for (int kb = 0; kb < KB; kb++) {
            const uint32_t qi = qc - KB + kb, qst = qi % QS;
            if (ok) ok = mbar_wait_bounded(smem_u32(sm.qfull + qst), (qi / QS) & 1, &sm.failed);
            if (!ok) break;
            tc_fence_after();
            const uint64_t qd = uniform64(smem_desc(base_u + at.q + qst * (NR * 128)));
#pragma unroll
            for (int kk = 0; kk < 4; kk++)
              mma_bf16_if(lead, dst, kd + kb * (kTcKeys * 8) + kk * 2, qd + kk * 2, p.idesc,
                          kb > 0 || kk > 0);
            if (!ONE) mma_commit_if(lead, smem_u32(sm.qempty + qst));
          }
          if (!ok) break;
          mma_commit_if(lead, smem_u32(sm.tfull + acc));
          if (i == todo - 1) mma_commit_if(lead, smem_u32(sm.kempty + kst));
        }
        kc += KG;
        q_unit = unit;
      }
      g += todo;
      if (g < run1) pos.next(a, p);
    }
    if (!ok) sm.failed = 1;
    __syncwarp();
  } else if (warp < kTcEpi) {
    // -------------------------------------------------------- epilogue
    const int wg = warp >> 2, quarter = warp & 3;
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const float zs = a.zscale;
    uint32_t qc = 0, jc = 0;
    int64_t q_unit = -1;
    int lo = 0;
    for (int64_t g = run0; g < run1 && ok;) {
      const int todo = (int)min((int64_t)max(pos.cnt, 1) - pos.off, run1 - g);
      const int64_t unit = (pos.l * a.n_req + pos.r) * a.H + pos.h;
      const int seq = a.seqused[pos.r];
      const int kt = ONE ? 0 : wg;
      const int p0 = (pos.kg * KG + kt) * kTcKeys, key = p0 + quarter * 32 + lane;
      const bool mine = ONE ? (jc & 1) == (uint32_t)wg : true;
      const bool whole = pos.off == 0 && todo == max(pos.cnt, 1);
      float *out = a.mass + unit * a.cap + key;
      float old = 0.f;
      // this thread's rows added up, keys lane/4 + 8·i of the warp's 32
      float s4[4] = {0.f, 0.f, 0.f, 0.f};
      int32_t blk = -1;
      if (mine && key < seq) {
        if (whole && key < a.n_mass[pos.r]) old = *out;
        blk = a.block_table[(int64_t)pos.r * a.max_blocks + page_of(key, a.bs_inv)];
      }
      if (pos.cnt > 0)
        for (int i = 0; i < todo && ok; i++) {
          if (!ONE || unit != q_unit) {  // another row tile
            if (ONE && qc > 0) {
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(sm.lempty + (qc - 1) % LS));
            }
            qc++;
            const int ls = (qc - 1) % LS;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.lfull + ls),
                                                           ((qc - 1) / LS) & 1, &sm.failed));
            if (!ok) break;
            lo = min(min(sm.lo[ls][0], sm.lo[ls][1]), min(sm.lo[ls][2], sm.lo[ls][3]));
            if (lo == INT_MAX) lo = 0;
          }
          const int ls = (qc - 1) % LS;
          const uint32_t job = ONE ? jc : jc + wg;
          jc += KG;
          if (mine) {
            const int acc = job % NACC;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.tfull + acc),
                                                           (job / NACC) & 1, &sm.failed));
            if (!ok) break;
            tc_fence_after();
            const uint32_t taddr = tmem + lane_base + acc * NR;
            const int qoff = ls * (NR + 16) + (lane & 3) * (NR / 4 + 4);
            const float *nl = reinterpret_cast<const float *>(base + at.nlse) + qoff;
            const int *vi = reinterpret_cast<const int *>(base + at.vis) + qoff;
            float t4[4] = {0.f, 0.f, 0.f, 0.f};  // this tile's, apart from the others'
            if (p0 + kTcKeys <= lo) {
              // every row sees every key of the tile
              uint32_t z[2][32];
              tmem_frag8(taddr, z[0]);
#pragma unroll 1
              for (int c = 0; c < NR; c += 64) {
                float n16[16];
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                  *reinterpret_cast<float4 *>(n16 + j) = *reinterpret_cast<const float4 *>(nl + c / 4 + j);
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                  tmem_wait(z[hf]);
                  if (hf == 0) tmem_frag8(taddr + c + (16u << 16), z[1]);
                  else if (c + 64 < NR) tmem_frag8(taddr + c + 64, z[0]);
#pragma unroll
                  for (int e = 0; e < 32; e += 4) {
                    const float w0 = ex2(fmaf(__uint_as_float(z[hf][e]), zs, n16[e / 2]));
                    const float w1 = ex2(fmaf(__uint_as_float(z[hf][e + 1]), zs, n16[e / 2 + 1]));
                    const float w2 = ex2(fmaf(__uint_as_float(z[hf][e + 2]), zs, n16[e / 2]));
                    const float w3 = ex2(fmaf(__uint_as_float(z[hf][e + 3]), zs, n16[e / 2 + 1]));
                    t4[2 * hf] += w0 + w1;
                    t4[2 * hf + 1] += w2 + w3;
                  }
                }
              }
            } else {
#pragma unroll 1
              for (int c = 0; c < NR; c += 64)
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                  uint32_t z[32];
                  tmem_frag8(taddr + c + ((uint32_t)(16 * hf) << 16), z);
                  tmem_wait(z);
                  const int k0 = p0 + quarter * 32 + hf * 16 + lane / 4;
#pragma unroll
                  for (int e = 0; e < 32; e++) {
                    const int col = c / 4 + (e >> 2) * 2 + (e & 1), k = k0 + 8 * ((e >> 1) & 1);
                    const float w = ex2(fmaf(__uint_as_float(z[e]), zs, nl[col]));
                    t4[2 * hf + ((e >> 1) & 1)] += k < vi[col] ? w : 0.f;
                  }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(sm.tempty + acc));
#pragma unroll
            for (int k = 0; k < 4; k++) s4[k] += t4[k];
          }
          if (!ONE) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(sm.lempty + ls));
          }
        }
      q_unit = unit;
      // the four lanes of a key, then each lane its own key
      float total_w = 0.f;
#pragma unroll
      for (int k = 0; k < 4; k++) {
        float x = s4[k];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
        x = __shfl_sync(0xFFFFFFFFu, x, (lane & 7) << 2);
        if ((lane >> 3) == k) total_w = x;
      }
      if (ok && mine) {
        const float add = blk >= 0 && blk < a.n_slots / a.BS ? total_w : 0.f;
        if (whole) {
          if (key < seq) *out = fmaf(a.decay, old, add);
        } else {
          p.part[(2 * (int64_t)blockIdx.x + (g != run0)) * (KG * kTcKeys) + kt * kTcKeys +
                 quarter * 32 + lane] = add;
        }
      }
      g += todo;
      if (g < run1) pos.next(a, p);
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
    for (int i = 0; i < KS; i++) {
      mbar_drain(smem_u32(sm.kfull + i), 0);
      mbar_drain(smem_u32(sm.kfull + i), 1);
    }
    for (int i = 0; i < QS; i++) {
      mbar_drain(smem_u32(sm.qfull + i), 0);
      mbar_drain(smem_u32(sm.qfull + i), 1);
    }
    for (int i = 0; i < NACC; i++) {
      mbar_drain(smem_u32(sm.tfull + i), 0);
      mbar_drain(smem_u32(sm.tfull + i), 1);
    }
  }
  __syncthreads();
  if (warp == kTcEpi + kTcProd) {
    tc_fence_after();
    free_tmem_cols(tmem, 512);
  }
}

// Row tiles of every key group of every request, one CTA per request.
__global__ void __launch_bounds__(256)
k_mass_plan(MassArgs a, MassTc p) {
  __shared__ int64_t sh[66];
  asm volatile("griddepcontrol.launch_dependents;");
  const int r = blockIdx.x, tid = threadIdx.x;
  int seq, r0, n;
  if (!mass_request(a, r, seq, r0, n)) {
    if (tid == 0) record_error(a.status, KVC_ERR_BOUNDS);
    return;
  }
  const int n_rt = (n + p.tokens - 1) / p.tokens;
  int *vis = p.rt_vis + (int64_t)r * p.max_rt;
  const int warp = tid >> 5, lane = tid & 31;
  for (int t = warp; t < n_rt; t += 8) {  // positions the widest row of each row tile sees
    const int i0 = t * p.tokens, i1 = min(n, i0 + p.tokens) - 1;
    int v = 0;
    for (int i = i0 + lane; i <= i1; i += 32) v = max(v, a.row_vis[r0 + i]);
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (lane == 0) vis[t] = min(v, seq);
  }
  __syncthreads();
  const int keys = 2 * kTcKeys, n_kg = (seq + keys - 1) / keys;
  int64_t *cum = p.cum + (int64_t)r * (p.max_kg + 1);
  int64_t carry = 0;
  for (int k0 = 0; k0 < n_kg; k0 += 256) {
    const int kg = k0 + tid;
    int64_t mine = 0;
    if (kg < n_kg) {
      int first = 0, last = n_rt - 1;
      while (first < n_rt && vis[first] <= kg * keys) first++;
      while (last >= first && vis[last] <= kg * keys) last--;
      const int cnt = last - first + 1;
      p.span[(int64_t)r * p.max_kg + kg] = make_int2(first, cnt);
      mine = max(cnt, 1);
    }
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    int64_t before = carry, tot = 0;
    for (int w = 0; w < 8; w++) {
      if (w < warp) before += sh[w];
      tot += sh[w];
    }
    if (kg < n_kg) cum[kg] = before + x - mine;
    carry += tot;
    __syncthreads();
  }
  if (tid == 0) cum[n_kg] = carry;
}

// CTA c: the group that the boundary before run c falls inside, if it is the
// first boundary inside that group.
__global__ void __launch_bounds__(256)
k_mass_join(MassArgs a, MassTc p) {
  __shared__ int64_t sh[66];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, c = blockIdx.x + 1;
  int64_t per = 0;
  for (int r = tid; r < a.n_req; r += 256) per += tc_request_work<false>(a, p, r);
  per = block_sum(per, sh);
  const int64_t total = per * a.L * a.H;
  const int n_cta = (int)min((int64_t)p.n_cta, total);
  if (c >= n_cta) return;
  const int64_t t = total * c / n_cta, prev = total * (c - 1) / n_cta;
  const TcPos<false> x = tc_find<false>(a, p, t, per, sh);
  if (x.off == 0) return;                 // the run begins with a group
  const int64_t g0 = t - x.off, g1 = g0 + max(x.cnt, 1);
  if (prev > g0) return;                  // an earlier boundary joins this group
  const int key = x.kg * 256 + tid, seq = a.seqused[x.r];
  if (key >= seq) return;
  // run c − 1 holds the group's beginning: its first part if it began there
  float sum = p.part[(2 * (int64_t)(c - 1) + (prev != g0)) * 256 + tid];
  for (int k = c; k < n_cta && total * k / n_cta < g1; k++) sum += p.part[2 * (int64_t)k * 256 + tid];
  float *out = a.mass + ((x.l * a.n_req + x.r) * a.H + x.h) * a.cap + key;
  *out = fmaf(a.decay, key < a.n_mass[x.r] ? *out : 0.f, sum);
}

// The shape of the tensor-core path for these sizes.
MassTc tc_plan(int n_req, int cap, int max_rows, int G, int D, bool &one, size_t &smem, size_t &ws,
               uint8_t *base) {
  MassTc p{};
  const int64_t R = (int64_t)max_rows * G;
  one = R <= 256;
  p.NR = R <= 128 ? 128 : 256;
  p.tokens = std::min(max_rows, p.NR / G);
  // what the row tiles leave: K tiles in flight when keys stream, else two
  const size_t tile = (size_t)kTcKeys * D * 2, q = (size_t)kTcQs * p.NR * 128;
  p.k_slots = one ? (int)std::min<size_t>(kTcMaxK, (200 * 1024 - q) / tile) & ~1 : 2;  // even: a slot keeps its MMA warp
  p.n_cta = device_sm_count();
  p.max_kg = (cap + 255) / 256;
  p.max_rt = (max_rows + p.tokens - 1) / p.tokens;
  p.idesc = make_idesc(128, p.NR);
  smem = 1024 + TcSmem(D, p.NR, p.k_slots, one ? 2 : 4).bytes;
  ws = 0;
  if (one) return p;
  auto take = [&](size_t n) {
    const size_t x = ws;
    ws += (n + 15) & ~size_t(15);
    return base + x;
  };
  p.cum = reinterpret_cast<int64_t *>(take((size_t)n_req * (p.max_kg + 1) * 8));
  p.span = reinterpret_cast<int2 *>(take((size_t)n_req * p.max_kg * 8));
  p.rt_vis = reinterpret_cast<int *>(take((size_t)n_req * p.max_rt * 4));
  p.part = reinterpret_cast<float *>(take((size_t)2 * p.n_cta * 256 * 4));
  return p;
}

template <class K, class... Args>
cudaError_t launch_dependent(K kern, dim3 grid, int threads, size_t smem, cudaStream_t s,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D>
cudaError_t launch_tc(const MassArgs &a, void *ws, cudaStream_t s) {
  bool one;
  size_t smem, ws_bytes;
  MassTc p = tc_plan(a.n_req, a.cap, a.max_rows, a.G, D, one, smem, ws_bytes,
                           reinterpret_cast<uint8_t *>(ws));
  auto *kern = one ? k_mass_tc<D, true> : k_mass_tc<D, false>;
  CUtensorMap tm_k{}, tm_q{};
  p.box = a.BS % 32 == 0 ? 32 : a.BS % 16 == 0 ? 16 : a.BS % 8 == 0 ? 8 : 0;
  if ((int64_t)a.L * a.n_slots > INT32_MAX) p.box = 0;  // (a map coordinate is an int32)
  p.q_box = !a.row_idx && (int64_t)a.L * a.n_q + a.n_rows <= INT32_MAX;
  if (p.box && !pool_map(&tm_k, a.kpool, (int64_t)a.L * a.n_slots, a.H, D, p.box))
    return cudaErrorUnknown;
  if (p.q_box && !q_map(&tm_q, a.q, (int64_t)a.L * a.n_q, a.Hq, D, a.G, p.tokens))
    return cudaErrorUnknown;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (one) {
    kern<<<p.n_cta, kTcThreads, smem, s>>>(tm_k, tm_q, a, p);
    return cudaGetLastError();
  }
  k_mass_plan<<<a.n_req, 256, 0, s>>>(a, p);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_dependent(kern, dim3(p.n_cta), kTcThreads, smem, s, tm_k, tm_q, a, p);
  if (e == cudaSuccess && p.n_cta > 1)
    e = launch_dependent(k_mass_join, dim3(p.n_cta - 1), 256, 0, s, a, p);
  return e;
}

}  // namespace

size_t attn_mass_ws_bytes(int n_req, int max_blocks, int max_rows, int, int H, int Hq, int D,
                          int BS) {
  if ((int64_t)max_rows * (Hq / H) <= kMrMaxRows) return 0;
  bool one;
  size_t smem, ws;
  tc_plan(n_req, max_blocks * BS, max_rows, Hq / H, D, one, smem, ws, nullptr);
  return ws;
}

cudaError_t launch_attn_mass(const uint16_t *q, const float *lse, int n_q,
                             const int32_t *row_idx, const int32_t *row_vis,
                             const int32_t *row_off, int n_rows, int max_rows,
                             const uint16_t *kpool, int64_t n_slots,
                             const int32_t *block_table, int max_blocks,
                             const int32_t *seqused, const int32_t *n_mass, int n_req, int L,
                             int H, int Hq, int D, int BS, float scale, float decay, float *mass,
                             void *ws, int32_t *status, cudaStream_t s) {
  MassArgs a{q,      kpool,   lse,    row_idx,  row_vis,    row_off,         block_table, seqused,
             n_mass, mass,    status, n_slots,  n_q,        n_rows,          max_rows,    max_blocks,
             max_blocks * BS, n_req,  L,        H,          Hq,              Hq / H,      BS,
             page_inverse(BS), scale * kLog2e, decay};
  const int64_t R = (int64_t)max_rows * a.G;
  if (R <= kMrMaxRows) {
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
  return D == 128 ? launch_tc<128>(a, ws, s) : launch_tc<64>(a, ws, s);
}

}  // namespace kvc
