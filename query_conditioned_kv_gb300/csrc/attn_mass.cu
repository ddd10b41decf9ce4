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
// warp: no atomics, and partial sums in memory only where a request has more
// rows than one row tile holds.
//
// k_mass_rows (few rows): bound by the stream of K, 2·D bytes per key.  All
// key tiles of all (layer, request, KV head) units, in order, are dealt out
// in equal contiguous runs to the CTAs; each of a CTA's four warps streams
// its 16 (D 128) or 32 (D 64) keys of a tile through a private cp.async ring
// (4 stages of 4 KB).  mma.sync m16n8k16, fp32 accumulators.  Measured: accepted
// paths of up to 6 nodes × 4 heads, 8 requests of 4K to 8K, 12 layers: 225 us,
// 5.5 TB/s, 83 % of a plain copy's rate.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>

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
// Widest row set (rows · G) of this path.  Both sides, 8 requests of 8K, 12
// layers, 24 rows: D 128 238 us here and 240 on the tensor cores, D 64 140 and
// 216; 32 rows, 512 positions of one request, 12 layers 13.2 and 13.1, 128K, four
// layers 193 and 185; 64 rows of a 128K window 322 and 178.
constexpr int kMrMaxRows = 32;
constexpr int kMrStages = 4;
constexpr int kMrStage = 4096;  // bytes of one warp's stage

template <int D, int NT>  // NT 8-row tiles of query rows
struct MassRowSmem {
  static constexpr int kRing = kMrWarps * kMrStages * kMrStage;
  static constexpr int kQ = kRing;
  static constexpr int kLse = kQ + NT * 8 * D * 2;  // lse·log2e per row
  static constexpr int kVis = kLse + NT * 8 * 4;    // positions each row sees
  static constexpr int kMisc = kVis + NT * 8 * 4;   // scratch [32] int64
  static constexpr int kValid = kMisc + 32 * 8;
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
  if (blockIdx.x == 0)  // one report per bad request
    for (int r = tid; r < a.n_req; r += kMrThreads) {
      int seq, r0, n;
      if (!mass_request(a, r, seq, r0, n)) record_error(a.status, KVC_ERR_BOUNDS);
    }
  auto tiles = [&](int x) { return (int64_t)mass_tiles(a, x, kTile); };
  const WarpSums sums = warp_sums(a.n_req, tiles);
  const int64_t per = sums.total;
  const int64_t total = per * a.L * a.H;
  const int n_cta = (int)min((int64_t)n_cta_max, total);
  if ((int)blockIdx.x >= n_cta) return;
  const int64_t run0 = div64(total * blockIdx.x, n_cta);
  const int64_t run1 = div64(total * (blockIdx.x + 1), n_cta);

  // run0 → (layer, request, head, tile): order l, r, h, tile.  H heads of a
  // request of w tiles: place x of a layer is place x / H of the sums, less what
  // the division drops.
  int64_t l = div64(run0, per * a.H), in_layer = run0 - l * per * a.H, before;
  int r;
  warp_find(sums, a.n_req, div64(in_layer, a.H), tiles, r, before);
  const int64_t in_request = in_layer - before * a.H;
  int n_kt = mass_tiles(a, r, kTile);
  int h = (int)div64(in_request, n_kt), t0 = (int)(in_request - (int64_t)h * n_kt);
  const int64_t n_blocks = a.n_slots / a.BS;

  for (int64_t g = run0; g < run1;) {
    int seq, r0, n;
    mass_request(a, r, seq, r0, n);
    const int t1 = (int)min((int64_t)n_kt, t0 + (run1 - g));
    const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
    const uint16_t *kl = a.kpool + (l * a.n_slots * a.H + h) * D;

    // block id of this lane's key, looked up a tile ahead of its copies
    int32_t blk = 0;
    auto look = [&](int t) {
      const int p = t * kTile + warp * KT + lane;
      if (lane < KT && p < seq) blk = bt[page_of(p, a.bs_inv)];
    };
    auto issue = [&](int t, int st) {
      const int p0 = t * kTile + warp * KT;
      int32_t slot = -1;
      if (lane < KT && p0 + lane < seq) {
        const int p = p0 + lane;
        if (blk >= 0 && blk < n_blocks) slot = blk * a.BS + p - page_of(p, a.bs_inv) * a.BS;
        else record_error(a.status, KVC_ERR_BOUNDS);
      }
      look(t + 1);
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
    look(t0);
#pragma unroll
    for (int s = 0; s < kMrStages - 1; s++) {
      if (t0 + s < t1) issue(t0 + s, s);
      cp_commit();
    }
    // this unit's rows: LSE and limits, then the queries.  A row that adds
    // nothing (past the request's rows, no limit, LSE ±inf) gets lse = +inf and
    // q = 0, so its weight is 0 wherever K is finite; `lo`, the least limit of
    // the others, tells the tiles that every one of them sees.
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
      // The tile's sums, with the rows' limits where some row stops inside or before
      // it.  An infinite key makes 0·inf = NaN in the rows that add nothing: sums
      // that are NaN are taken again with the limits, which leave those rows out.
      float sum[MT][2];
      for (bool masked = p0 + KT > lo;; masked = true) {
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
        bool nan = false;
#pragma unroll
        for (int mt = 0; mt < MT; mt++) nan |= sum[mt][0] != sum[mt][0] || sum[mt][1] != sum[mt][1];
        if (masked || !__any_sync(0xFFFFFFFFu, nan)) break;
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
  static std::atomic<int> cached{0};  // (a property of the kernel; the query takes as long as a launch)
  int per_sm = cached.load(std::memory_order_relaxed);
  if (!per_sm) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_mass_rows<D, NT>, kMrThreads, smem);
    if (e != cudaSuccess) return e;
    cached.store(per_sm, std::memory_order_relaxed);
  }
  constexpr int tile = kMrWarps * 2048 / D;
  const int64_t most = (int64_t)a.L * a.n_req * a.H * ((a.cap + tile - 1) / tile);
  const int n_cta = (int)std::min<int64_t>((int64_t)std::min(per_sm, 3) * device_sm_count(), most);
  k_mass_rows<D, NT><<<n_cta, kMrThreads, smem, s>>>(a, n_cta);
  return cudaGetLastError();
}

// --------------------------------------------------------------- many rows
//
// tcgen05: D[key][row] = K tile (M 128 keys, A) × row tile (N rows, B), fp32 in
// tensor memory.  The rows stay in shared memory while the keys stream past.
// Warps 0–15: two epilogue groups of eight; 16–19: producers; then the
// products' issuers (RT = 1: a warp for each group, so that a warp's waits run
// under the other's products; RT = 2: one, in order, as two warps' products
// would interleave and both end late) and a warp for the rows' TMA boxes.  An epilogue thread owns two keys and a quarter of
// the rows (16x256b fragments): the rows' LSE, stored in that order, costs it
// half of the shared-memory reads that one key a thread would.
//
// RT = 1 (a request's rows fit one row tile): the key tiles alternate between
// the groups, and a tile's sums go straight into `mass`.
// RT = 2: a unit is a pair of row tiles, one for each group, with the keys
// that some row of it sees (under a causal limit, half of them); every row
// tile writes its sums to the workspace, and k_mass_join adds them in order.
// Streaming the rows past resident keys instead moves 64 KB per two products
// where this moves 32 KB, and could not be kept ahead of the tensor core
// (measured: 2080 cycles a product against 1008).
//
// Bound: RT = 1 the K stream (32 rows × 4 heads over 128K, four layers: 191 us,
// 5.8 TB/s, 87 % of a plain copy's rate); RT = 2 the products (1008 cycles per 128
// keys × 256 rows) and the ex2s (1024), which cannot all overlap, for tensor
// memory holds two accumulators of 256 columns: 8192 causal rows × 4 heads 326 us,
// 845 TFLOP/s.  Four accumulators of 128 columns took 349 us (an instruction of
// half the columns takes 105 cycles of 126), eight epilogue warps 337.
//
// Work is dealt out by key tile in equal contiguous runs, one per CTA.

constexpr int kTcEpi = 16;                      // epilogue warps, half for each accumulator
constexpr int kTcProd = 4;                      // producer warps
constexpr int kTcThreads = (kTcEpi + kTcProd + 4) * 32;  // (the last warps idle)
// Registers a thread after setmaxnreg: what the launch holds, 768 · 80, split
// 512 · 88 + 256 · 64.
constexpr int kTcMore = 88, kTcLess = 64;
constexpr int kTcKeys = 128;                    // keys of a tile
constexpr int kTcMaxK = 8;                      // K slots, at most
constexpr size_t kTcSmemMax = 232448;           // of a CTA
constexpr size_t kTcPartBytes = size_t(1) << 29;  // partial sums of one launch, about

struct MassTc {
  int n_cta;        // CTAs the work is dealt out to
  int NR;           // rows of a row tile's buffers: 128 or 256
  int tokens;       // rows i (tokens) of a row tile: tokens·G ≤ NR rows
  int k_slots;      // K ring
  int box;          // rows of a TMA box of K (a divisor of the page size), 0: none
  int q_box;        // queries by TMA (no row_idx)
  int rg0, n_rg;    // RT 2: this launch's pairs of row tiles, [rg0, rg0 + n_rg)
  uint32_t idesc;
  int64_t *cum;     // [n_req][n_rg + 1]: key tiles before each pair
  int64_t cap4;     // cap rounded up to whole float4
  float *part;      // [L·n_req·H][2·n_rg][cap4]: each row tile's sums
};

// Head of the dynamic shared memory (fixed offsets), behind K and q; then the
// LSE slots: −lse·log2e, [slot][NR + 16] in the order of lse_at.
struct TcHead {
  uint64_t kfull[kTcMaxK], kempty[kTcMaxK], qfull[2], qempty[2], lfull[2], lempty[2];
  uint64_t tfull[4], tempty[4];
  int64_t run[2], at_l;  // the CTA's run of tiles, and where it begins
  int at[5];
  int lo[2][4];  // least limit of the slot's rows, per producer warp
  uint32_t tmem_holder;
  volatile int failed;
};
constexpr uint32_t kTcHead = 384;
static_assert(sizeof(TcHead) <= kTcHead, "the head's room");

struct TcSmem {
  uint32_t q, head, nlse, bytes;  // K at 0
  __host__ __device__ TcSmem(int D, int NR, int ks) {
    q = ks * kTcKeys * D * 2;
    head = q + 2 * NR * D * 2;
    nlse = head + kTcHead;
    bytes = nlse + 2 * (NR + 16) * 4;
  }
};

// Place of row r in an LSE slot: the rows 8k + 2q + {0, 1} of an epilogue
// thread (q = lane mod 4) together, quarters four words apart in the banks.
__device__ __forceinline__ int lse_at(int r, int NR) {
  return ((r >> 1) & 3) * (NR / 4 + 4) + (r >> 3) * 2 + (r & 1);
}

// Key tiles of request r, per layer and head.
template <int RT>
__device__ __forceinline__ int64_t tc_request_work(const MassArgs &a, const MassTc &p, int r) {
  return RT == 1 ? mass_tiles(a, r, kTcKeys) : p.cum[(int64_t)r * (p.n_rg + 1) + p.n_rg];
}

// Where a run stands: key tile t of unit (l, r, h, pair rg), n_t tiles in it.
template <int RT>
struct TcPos {
  int64_t l;
  int r, h, rg, t, n_t;
  __device__ __forceinline__ void pair(const MassArgs &a, const MassTc &p) {
    if (RT == 1) {
      n_t = mass_tiles(a, r, kTcKeys);
    } else {
      const int64_t *c = p.cum + (int64_t)r * (p.n_rg + 1) + rg;
      n_t = (int)(c[1] - c[0]);
    }
  }
  // the next tile (one exists while the run is not over)
  __device__ __forceinline__ void next(const MassArgs &a, const MassTc &p) {
    if (++t < n_t) return;
    t = 0;
    do {
      if (++rg == (RT == 1 ? 1 : p.n_rg)) {
        rg = 0;
        if (++h == a.H) {
          h = 0;
          if (++r == a.n_req) {
            r = 0;
            l++;
          }
        }
      }
      pair(a, p);
    } while (n_t == 0);
  }
  __device__ __forceinline__ int64_t unit(const MassArgs &a) const {
    return (l * a.n_req + r) * a.H + h;
  }
};

// Position of tile x; sums: of the requests' tiles per layer and head.
template <int RT>
__device__ __forceinline__ TcPos<RT> tc_find(const MassArgs &a, const MassTc &p, int64_t x,
                                             const WarpSums &sums) {
  TcPos<RT> f;
  const int64_t layer = sums.total * a.H;
  f.l = div64(x, layer);
  int64_t before;
  const int64_t in_layer = x - f.l * layer;
  warp_find(
      sums, a.n_req, div64(in_layer, a.H), [&](int r) { return tc_request_work<RT>(a, p, r); }, f.r,
      before);
  before *= a.H;
  const int64_t w = tc_request_work<RT>(a, p, f.r);
  f.h = (int)div64(in_layer - before, w);
  const int64_t in_head = in_layer - before - f.h * w;
  if (RT == 1) {
    f.rg = 0;
    f.t = (int)in_head;
  } else {
    const int64_t *cum = p.cum + (int64_t)f.r * (p.n_rg + 1);
    int lo = 0, hi = p.n_rg - 1;  // the last pair with cum ≤ in_head
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= in_head) lo = mid;
      else hi = mid - 1;
    }
    f.rg = lo;
    f.t = (int)(in_head - cum[lo]);
  }
  f.pair(a, p);
  return f;
}

template <int D, int RT>
__global__ void __launch_bounds__(kTcThreads, 1)
k_mass_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
          MassArgs a, MassTc p) {
  constexpr int CH = D / 8, KB = D / 64;
  constexpr uint32_t kSlot = kTcKeys * D * 2;
  constexpr int kMma = RT == 1 ? 2 : 1;  // MMA warps
  extern __shared__ __align__(1024) uint8_t base[];
  const int NR = p.NR, KS = p.k_slots, NACC = 512 / NR;
  const TcSmem at(D, NR, KS);
  TcHead &sm = *reinterpret_cast<TcHead *>(base + at.head);
  float *nlse = reinterpret_cast<float *>(base + at.nlse);
  const uint32_t base_u = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (RT == 2) asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
  if (warp == 0) {
    const WarpSums sums = warp_sums(a.n_req, [&](int r) { return tc_request_work<RT>(a, p, r); });
    const int64_t total = sums.total * a.L * a.H;
    const int n_cta = (int)min((int64_t)p.n_cta, total);
    // (a misaligned base cannot hold swizzled tiles: nothing would be right)
    const bool works = (int)blockIdx.x < n_cta && (base_u & 1023u) == 0;
    if ((base_u & 1023u) != 0 && lane == 0) record_error(a.status, KVC_ERR_CUDA);
    TcPos<RT> f{};
    int64_t run0 = 0, run1 = 0;
    if (works) {
      run0 = div64(total * blockIdx.x, n_cta);
      run1 = div64(total * (blockIdx.x + 1), n_cta);
      f = tc_find<RT>(a, p, run0, sums);
    }
    if (lane == 0) {
      sm.run[0] = run0;
      sm.run[1] = run1;
      sm.at_l = f.l;
      sm.at[0] = f.r;
      sm.at[1] = f.h;
      sm.at[2] = f.rg;
      sm.at[3] = f.t;
      sm.at[4] = f.n_t;
    }
  } else if (warp == 1 && lane == 0) {
    sm.failed = 0;
    for (int i = 0; i < KS; i++) {
      mbar_init(smem_u32(sm.kfull + i), kTcProd * 32);
      mbar_init(smem_u32(sm.kempty + i), 1);
    }
    for (int i = 0; i < 2; i++) {
      // RT 1: both MMA warps and both epilogue groups use a unit's rows;
      // RT 2: slot i is group i's
      mbar_init(smem_u32(sm.qfull + i), p.q_box ? 1 : kTcProd * 32);
      mbar_init(smem_u32(sm.qempty + i), kMma);
      mbar_init(smem_u32(sm.lfull + i), kTcProd * 32);
      mbar_init(smem_u32(sm.lempty + i), RT == 1 ? kTcEpi : kTcEpi / 2);
    }
    for (int i = 0; i < NACC; i++) {
      mbar_init(smem_u32(sm.tfull + i), 1);
      mbar_init(smem_u32(sm.tempty + i), kTcEpi / 2);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows that no row tile fills stay zero
  if (p.tokens * a.G < NR) {
    for (uint32_t i = tid; i < 2u * NR * D * 2 / 16; i += kTcThreads)
      *reinterpret_cast<uint4 *>(base + at.q + i * 16) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kTcEpi + kTcProd) alloc_tmem_cols(&sm.tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_holder;

  if (RT == 1 && blockIdx.x == 0)  // one report per bad request
    for (int r = tid; r < a.n_req; r += kTcThreads) {
      int seq, r0, n;
      if (!mass_request(a, r, seq, r0, n)) record_error(a.status, KVC_ERR_BOUNDS);
    }
  const int64_t run0 = sm.run[0], run1 = sm.run[1];
  TcPos<RT> pos{sm.at_l, sm.at[0], sm.at[1], sm.at[2], sm.at[3], sm.at[4]};
  if (RT == 2) asm volatile("griddepcontrol.launch_dependents;");

  bool ok = true;
  uint32_t uc = 0;    // units begun
  if (warp >= kTcEpi && warp < kTcEpi + kTcProd) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcLess));
    // ------------------------------------------------------- producers
    // K: 32 keys of a tile a warp, by TMA boxes of whole page rows or row by row
    // with cp.async (bad blocks, the end, page sizes without a box).  Rows: by
    // another warp's TMA boxes, or row by row here, through row_idx; their LSE
    // here.
    const int pw = warp - kTcEpi;
    const int64_t n_blocks = a.n_slots / a.BS;
    constexpr int RPI = 32 / CH;
    const int col = lane % CH;
    uint32_t kc = 0;                // K tiles loaded
    uint32_t pend0 = 0, pend1 = 0;  // stages copied by cp.async and not handed over, oldest first
    int32_t blk = 0;                // block id of this lane's key of the next tile
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
    // this lane's rows of a row tile: 32·pw + 128·u + lane
    const int tok0 = (32 * pw + lane) / a.G, g0 = (32 * pw + lane) % a.G;
    const int tok1 = (32 * pw + lane + 128) / a.G, g1 = (32 * pw + lane + 128) % a.G;
    for (int64_t g = run0; g < run1 && ok; g++) {
      int seq, r0, n;
      mass_request(a, pos.r, seq, r0, n);
      const int32_t *bt = a.block_table + (int64_t)pos.r * a.max_blocks;
      const bool begins = g == run0 || pos.t == 0;  // of a unit, in this run
      auto look = [&](int t) {
        const int pp = t * kTcKeys + pw * 32 + lane;
        blk = pp < seq ? bt[page_of(pp, a.bs_inv)] : 0;
      };
      if (begins) look(pos.t);
      // ---- the tile of K
      const int pp = pos.t * kTcKeys + pw * 32 + lane;
      int32_t slot = -1;
      if (pp < seq) {
        if (blk >= 0 && blk < n_blocks) slot = blk * a.BS + pp - page_of(pp, a.bs_inv) * a.BS;
        else record_error(a.status, KVC_ERR_BOUNDS);
      }
      look(pos.t + 1);
      const uint32_t st = kc % KS;
      if (!(ok = acquire(sm.kempty + st, ((kc / KS) & 1) ^ 1))) break;
      kc++;
      const uint32_t bar = smem_u32(sm.kfull + st);
      const uint32_t slot0 = base_u + st * kSlot + pw * 32 * 128;
      if (p.box > 0 && __all_sync(0xFFFFFFFFu, slot >= 0)) {
        if (lane == 0) mbar_expect_tx(bar, kSlot / kTcProd);
        else mbar_arrive(bar);
        __syncwarp();
        // (warp-uniform operands, one lane enabled)
        const uint32_t ubar = uniform32(bar), udst = uniform32(slot0), uh = uniform32(pos.h);
        const uint32_t row0 = uniform32((uint32_t)(pos.l * a.n_slots));
        for (int k = 0; k < 32; k += p.box) {
          const uint32_t sl = __shfl_sync(0xFFFFFFFFu, slot, k);
#pragma unroll
          for (int kb = 0; kb < KB; kb++)
            tma_load_3d_if(lane == 0, udst + k * 128 + kb * (kTcKeys * 128), &tm_k, kb * 64, uh,
                           row0 + sl, ubar);
        }
      } else {
        const uint16_t *kl = a.kpool + (pos.l * a.n_slots * a.H + pos.h) * D;
        const uint32_t dst = slot0 + (col >> 3) * (kTcKeys * 128);
#pragma unroll 4
        for (int i = 0; i < 32 / RPI; i++) {
          const int row = i * RPI + lane / CH;
          const int32_t sl = __shfl_sync(0xFFFFFFFFu, slot, row);
          cp_async16(dst + row * 128 + (((col & 7) ^ (row & 7)) << 4),
                     kl + (int64_t)max(sl, 0) * a.H * D + col * 8, sl >= 0);
        }
        committed(bar);
      }
      // ---- a new unit's rows
      if (begins) {
        const float *lse = a.lse + pos.l * a.n_q * a.Hq + pos.h * a.G;
#pragma unroll 1
        for (int j = 0; j < RT && ok; j++) {
          const uint32_t s = RT == 1 ? uc & 1 : j, use = RT == 1 ? uc >> 1 : uc;
          const int rt = RT == 1 ? 0 : 2 * (p.rg0 + pos.rg) + j;
          if (!(ok = acquire(sm.lempty + s, (use & 1) ^ 1))) break;
          // A row that adds nothing (past the request's rows, no limit, LSE ±inf)
          // has weight 0 by its LSE where its product is finite: its query is
          // zeros, or, where a box brought it along and it may be anything, the
          // tiles are masked for every key (lo = 0).
          int lo = INT_MAX;
          int64_t src_row[2];
#pragma unroll
          for (int u = 0; u < 2; u++) {
            src_row[u] = -1;
            if (u == 1 && NR == 128) break;
            const int tok = u ? tok1 : tok0, i = rt * p.tokens + tok;
            float nl = -INFINITY;
            if (tok < p.tokens) {
              if (i < n) {
                const int vis = min(a.row_vis[r0 + i], seq), x = a.row_idx ? a.row_idx[r0 + i] : r0 + i;
                if (vis > 0 && x >= 0 && x < a.n_q) {
                  const float l2 = lse[(int64_t)x * a.Hq + (u ? g1 : g0)] * kLog2e;
                  if (fabsf(l2) != INFINITY) {
                    nl = -l2;
                    lo = min(lo, vis);
                    src_row[u] = (pos.l * a.n_q + x) * a.Hq + pos.h * a.G + (u ? g1 : g0);
                  }
                } else if (vis > 0) {
                  record_error(a.status, KVC_ERR_BOUNDS);
                }
              }
              if (p.q_box && nl == -INFINITY) lo = 0;
            }
            nlse[s * (NR + 16) + lse_at(128 * u + 32 * pw + lane, NR)] = nl;
          }
          lo = __reduce_min_sync(0xFFFFFFFFu, lo);
          if (lane == 0) sm.lo[s][pw] = lo;
          __syncwarp();
          mbar_arrive(smem_u32(sm.lfull + s));
          if (p.q_box) continue;
          if (!(ok = acquire(sm.qempty + s, (use & 1) ^ 1))) break;
          const uint32_t dst = base_u + at.q + s * (NR * D * 2) + (col >> 3) * (NR * 128);
#pragma unroll
          for (int u = 0; u < 2; u++) {
            if (u == 1 && NR == 128) break;
#pragma unroll 4
            for (int i = 0; i < 32 / RPI; i++) {
              const int rr = i * RPI + lane / CH;
              const int64_t src = __shfl_sync(0xFFFFFFFFu, src_row[u], rr);
              cp_async16(dst + (128 * u + 32 * pw + rr) * 128 + (((col & 7) ^ (rr & 7)) << 4),
                         a.q + max(src, (int64_t)0) * D + col * 8, src >= 0);
            }
          }
          committed(smem_u32(sm.qfull + s));
        }
        flush();  // (the next stages may all be boxes)
        uc++;
      }
      if (g + 1 < run1) pos.next(a, p);
    }
    flush();
    cp_wait<0>();
    if (!ok) sm.failed = 1;
  } else if (warp >= kTcEpi + kTcProd) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcLess));
    if (warp == kTcEpi + kTcProd + kMma) {
      // ----------------------------------------------- rows by TMA boxes
      if (p.q_box && lane == 0)
        for (int64_t g = run0; g < run1 && ok; g++) {
          if (g == run0 || pos.t == 0) {
            for (int j = 0; j < RT && ok; j++) {
              const uint32_t s = RT == 1 ? uc & 1 : j, use = RT == 1 ? uc >> 1 : uc;
              const int rt = RT == 1 ? 0 : 2 * (p.rg0 + pos.rg) + j;
              const uint32_t bar = smem_u32(sm.qfull + s);
              if (!(ok = mbar_wait_bounded(smem_u32(sm.qempty + s), (use & 1) ^ 1, &sm.failed))) break;
              mbar_expect_tx(bar, p.tokens * a.G * D * 2);
  #pragma unroll
              for (int kb = 0; kb < KB; kb++)
                tma_load_3d(base_u + at.q + s * (NR * D * 2) + kb * (NR * 128), &tm_q, kb * 64,
                            pos.h * a.G, (int)(pos.l * a.n_q) + a.row_off[pos.r] + rt * p.tokens, bar);
            }
            uc++;
          }
          if (g + 1 < run1) pos.next(a, p);
        }
      if (!ok) sm.failed = 1;
      __syncwarp();
    } else if (warp < kTcEpi + kTcProd + kMma) {
      // ----------------------------------------------------- MMA issuers
      // (the whole warp runs the loop; one lane's products are enabled)
      const uint32_t wg = warp - kTcEpi - kTcProd;  // RT 1: the group it works for
      const uint32_t lead = lane == 0;
      uint32_t kc = 0;  // K tiles
      uint64_t qd[2] = {0, 0};
      for (int64_t g = run0; g < run1 && ok; g++, kc++) {
        if (g == run0 || pos.t == 0) {
          if (uc > 0) {
#pragma unroll
            for (int j = 0; j < RT; j++)
              mma_commit_if(lead, smem_u32(sm.qempty + (RT == 1 ? (uc - 1) & 1 : j)));
          }
          uc++;
        }
        const uint32_t st = kc % KS;
        const uint64_t kd = uniform64(smem_desc(base_u + st * kSlot));
        const bool mine = RT == 2 || (kc & 1) == wg;
#pragma unroll
        for (int j = 0; j < RT; j++) {
          // (RT 1: also for a unit without a tile of this warp's: a barrier's parity
          // tells only two uses apart)
          if (g == run0 || pos.t == 0) {
            const uint32_t s = RT == 1 ? (uc - 1) & 1 : j, use = RT == 1 ? (uc - 1) >> 1 : uc - 1;
            if (!(ok = mbar_wait_bounded(smem_u32(sm.qfull + s), use & 1, &sm.failed))) break;
            qd[j] = uniform64(smem_desc(base_u + at.q + s * (NR * D * 2)));
          }
          const uint32_t acc = RT == 2 ? j : kc % NACC, use = RT == 2 ? kc : kc / NACC;
          if (!mine) break;
          if (j == 0) ok = mbar_wait_bounded(smem_u32(sm.kfull + st), (kc / KS) & 1, &sm.failed);
          if (ok) ok = mbar_wait_bounded(smem_u32(sm.tempty + acc), (use & 1) ^ 1, &sm.failed);
          if (!ok) break;
          tc_fence_after();
          const uint32_t dst = uniform32(tmem + acc * NR), qk = uniform32(NR * 8);
#pragma unroll
          for (int kk = 0; kk < 4 * KB; kk++)
            mma_bf16_if(lead, dst, kd + (kk >> 2) * (kTcKeys * 8) + (kk & 3) * 2,
                        qd[j] + (kk >> 2) * qk + (kk & 3) * 2, p.idesc, kk > 0);
          mma_commit_if(lead, smem_u32(sm.tfull + acc));
        }
        if (!ok) break;
        if (mine) mma_commit_if(lead, smem_u32(sm.kempty + st));
        if (g + 1 < run1) pos.next(a, p);
      }
      if (!ok) sm.failed = 1;
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcMore));
    // -------------------------------------------------------- epilogue
    const int wg = warp >> 3, quarter = warp & 3, half = (warp >> 2) & 1;
    const int key0 = quarter * 32 + half * 16;  // the warp's 16 keys of a tile
    const uint32_t lane_base = (uint32_t)key0 << 16;
    const int my_key = key0 + lane / 4 + 8 * (lane & 1);  // the one this lane writes (lane & 2: none)
    const uint64_t zs2 = pk2(a.zscale, a.zscale);
    uint32_t kc = 0, jc = 0;
    int lo = 0;
    const float *nl = nlse;  // the slot's LSE
    const int nl_q = (lane & 3) * (NR / 4 + 4);
    const int64_t n_blocks = a.n_slots / a.BS;
    // the lane's key: its sum's place, its block id and its weight so far, the
    // last two fetched a tile of the group ahead
    constexpr int kStep = RT == 1 ? 2 * kTcKeys : kTcKeys;
    int seq = 0, n_old = 0;
    float *out0 = nullptr, old = 0.f, next_old = 0.f;
    const int32_t *bt = nullptr;
    int32_t blk = -1, next_blk = -1;
    auto fetch = [&](int key) {
      next_blk = key < seq ? bt[page_of(key, a.bs_inv)] : -1;
      if (RT == 1) next_old = key < n_old ? out0[key] : 0.f;
    };
    for (int64_t g = run0; g < run1 && ok; g++, kc++) {
      const bool mine = RT == 2 || (kc & 1) == (uint32_t)wg;
      const int p0 = pos.t * kTcKeys, key = p0 + my_key;
      if (g == run0 || pos.t == 0) {
        __syncwarp();
        if (uc > 0 && lane == 0) mbar_arrive(smem_u32(sm.lempty + (RT == 1 ? (uc - 1) & 1 : wg)));
        const int64_t u = pos.unit(a);
        seq = a.seqused[pos.r];
        bt = a.block_table + (int64_t)pos.r * a.max_blocks;
        if (RT == 1) n_old = min(seq, a.n_mass[pos.r]);
        out0 = RT == 1 ? a.mass + u * a.cap : p.part + (u * 2 * p.n_rg + 2 * pos.rg + wg) * p.cap4;
        fetch(mine ? key : key + kTcKeys);
        const uint32_t s = RT == 1 ? uc & 1 : wg, use = RT == 1 ? uc >> 1 : uc;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.lfull + s), use & 1, &sm.failed));
        if (!ok) break;
        lo = min(min(sm.lo[s][0], sm.lo[s][1]), min(sm.lo[s][2], sm.lo[s][3]));
        if (lo == INT_MAX) lo = 0;
        nl = nlse + s * (NR + 16);
        uc++;
      }
      if (mine) {
        const uint32_t acc = RT == 2 ? wg : kc % NACC, use = RT == 2 ? jc : kc / NACC;
        blk = next_blk;
        old = next_old;
        fetch(key + kStep);
        ok = __all_sync(0xFFFFFFFFu,
                        mbar_wait_bounded(smem_u32(sm.tfull + acc), use & 1, &sm.failed));
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + lane_base + acc * NR;
        uint64_t s2[2] = {0, 0};  // keys lane/4 and lane/4 + 8, even and odd rows
        bool masked = p0 + kTcKeys > lo;
        if (!masked) {
          // every row sees every key of the tile
          uint32_t z[2][16];
          tmem_frag4(taddr, z[0]);
#pragma unroll 1
          for (int c = 0; c < NR; c += 64) {
            uint64_t t2[2] = {0, 0};
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
              float n8[8];
#pragma unroll
              for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<float4 *>(n8 + j) =
                    *reinterpret_cast<const float4 *>(nl + nl_q + c / 4 + 8 * hf + j);
              tmem_wait(z[hf]);
              if (hf == 0 || c + 64 < NR) tmem_frag4(taddr + c + 32 * hf + 32, z[hf ^ 1]);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const int j = (e >> 2) * 2;
                float w0, w1;
                upk2(fma2(pk2(__uint_as_float(z[hf][e]), __uint_as_float(z[hf][e + 1])), zs2,
                          pk2(n8[j], n8[j + 1])),
                     w0, w1);
                t2[(e >> 1) & 1] = add2(t2[(e >> 1) & 1], pk2(ex2(w0), ex2(w1)));
              }
            }
            s2[0] = add2(s2[0], t2[0]);
            s2[1] = add2(s2[1], t2[1]);
          }
          // an infinite key is NaN in the rows that add nothing (0·inf): the sums
          // again, without those rows
          float x, y;
          upk2(add2(s2[0], s2[1]), x, y);
          masked = __any_sync(0xFFFFFFFFu, x + y != x + y);
        }
        if (masked) {
          // the rows' limits: 32 rows a lane-wide load, one exchange per two rows
          const int r0 = a.row_off[pos.r], n = a.row_off[pos.r + 1] - r0;
          const int i0 = RT == 1 ? 0 : (2 * (p.rg0 + pos.rg) + wg) * p.tokens;
          const int k0 = p0 + key0 + lane / 4;
          float m0 = 0.f, m1 = 0.f;
#pragma unroll 1
          for (int c = 0; c < NR; c += 32) {
            uint32_t z[16];
            tmem_frag4(taddr + c, z);
            const int i = i0 + (c + lane) / a.G;
            int vis = 0;
            if (i < n && nl[lse_at(c + lane, NR)] != -INFINITY) vis = a.row_vis[r0 + i];
            tmem_wait(z);
#pragma unroll
            for (int e = 0; e < 16; e += 4)
#pragma unroll
              for (int b = 0; b < 2; b++) {
                const int v = __shfl_sync(0xFFFFFFFFu, vis, 2 * e + 2 * (lane & 3) + b);
                const float nb = nl[nl_q + c / 4 + e / 2 + b];
                const float w0 = ex2(fmaf(__uint_as_float(z[e + b]), a.zscale, nb));
                const float w1 = ex2(fmaf(__uint_as_float(z[e + 2 + b]), a.zscale, nb));
                m0 += k0 < v ? w0 : 0.f;
                m1 += k0 + 8 < v ? w1 : 0.f;
              }
          }
          s2[0] = pk2(m0, 0.f);
          s2[1] = pk2(m1, 0.f);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(sm.tempty + acc));
        // the four lanes of two keys: each pair of lanes keeps one key
        float x, y, sum, away;
        upk2(s2[0], x, y);
        sum = x + y;
        upk2(s2[1], x, y);
        away = x + y;
        if (lane & 1) {
          const float h = sum;
          sum = away;
          away = h;
        }
        sum += __shfl_xor_sync(0xFFFFFFFFu, away, 1);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
        if (blk < 0 || blk >= n_blocks) sum = 0.f;
        if (key < seq && !(lane & 2)) out0[key] = RT == 1 ? fmaf(a.decay, old, sum) : sum;
        jc++;
      }
      if (g + 1 < run1) pos.next(a, p);
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
    for (int i = 0; i < 2; i++) {
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

// Key tiles of each pair of row tiles (up to the widest limit among its rows)
// and their running sums, one CTA per request.
__global__ void __launch_bounds__(256)
k_mass_plan(MassArgs a, MassTc p) {
  __shared__ int64_t sh[64];
  asm volatile("griddepcontrol.launch_dependents;");
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t *cum = p.cum + (int64_t)r * (p.n_rg + 1);
  int seq, r0, n;
  const bool ok = mass_request(a, r, seq, r0, n);
  if (!ok && tid == 0) record_error(a.status, KVC_ERR_BOUNDS);
#pragma unroll 4
  for (int rg = warp; rg < p.n_rg; rg += 8) {
    int v = 0;
    if (ok) {
      const int64_t i0 = (int64_t)2 * (p.rg0 + rg) * p.tokens;
      const int i1 = (int)min((int64_t)n, i0 + 2 * p.tokens);
      for (int64_t i = i0 + lane; i < i1; i += 32) v = max(v, min(a.row_vis[r0 + i], seq));
    }
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (lane == 0) cum[rg + 1] = (v + kTcKeys - 1) / kTcKeys;
  }
  __syncthreads();
  int64_t carry = 0;
  for (int k0 = 0; k0 < p.n_rg; k0 += 256) {
    const int rg = k0 + tid;
    const int64_t mine = rg < p.n_rg ? cum[rg + 1] : 0;
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
    if (rg < p.n_rg) cum[rg + 1] = before + x;
    carry += tot;
    __syncthreads();
  }
  if (tid == 0) cum[0] = 0;
}

// The row tiles' sums added up, on top of what is there (the first launch's: the
// decayed weight): warp w takes the pairs w, w + 8, …, then the warps' sums are
// added in order.  blockIdx.x: a key tile, y · z: unit.
__global__ void __launch_bounds__(256)
k_mass_join(MassArgs a, MassTc p) {
  static_assert(kTcKeys == 128, "a float4 a lane");
  __shared__ float4 sh[8][32];
  const int64_t unit = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (unit >= (int64_t)a.L * a.n_req * a.H) return;
  const int r = (int)(unit / a.H % a.n_req);
  int seq, r0, n;
  if (!mass_request(a, r, seq, r0, n) || t * kTcKeys >= seq) return;
  const int64_t *cum = p.cum + (int64_t)r * (p.n_rg + 1);
  const float *part = p.part + unit * 2 * p.n_rg * p.cap4 + t * kTcKeys + 4 * lane;
  const bool in = t * kTcKeys + 4 * lane < p.cap4;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int rg = warp; rg < p.n_rg; rg += 8)
    if (in && t < (int)(cum[rg + 1] - cum[rg])) {
      const float *x = part + (int64_t)2 * rg * p.cap4;
      const float4 u = *reinterpret_cast<const float4 *>(x);
      const float4 v = *reinterpret_cast<const float4 *>(x + p.cap4);
      sum.x += u.x + v.x;
      sum.y += u.y + v.y;
      sum.z += u.z + v.z;
      sum.w += u.w + v.w;
    }
  sh[warp][lane] = sum;
  __syncthreads();
  const int key = t * kTcKeys + threadIdx.x;
  if (threadIdx.x >= kTcKeys || key >= seq) return;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < 8; w++) s += reinterpret_cast<const float *>(sh[w])[threadIdx.x];
  float *out = a.mass + unit * a.cap + key;
  if (p.rg0 == 0) *out = fmaf(a.decay, key < a.n_mass[r] ? *out : 0.f, s);
  else *out += s;
}

// The shape of the tensor-core path for these sizes; n_rg pairs of row tiles a
// launch when they do not fit one tile.
MassTc tc_plan(int n_req, int cap, int max_rows, int L, int H, int G, int D, int &pairs,
               size_t &smem, size_t &ws, uint8_t *base) {
  MassTc p{};
  const int64_t R = (int64_t)max_rows * G;
  const bool one = R <= 256;
  p.NR = R <= 128 ? 128 : 256;
  p.tokens = std::min(max_rows, p.NR / G);
  // K tiles in flight: what the two row tiles leave.  Even for RT 1, so that a
  // slot's tiles are all one MMA warp's.
  p.k_slots = kTcMaxK;
  while (p.k_slots > 2 && (TcSmem(D, p.NR, p.k_slots).bytes > kTcSmemMax || (one && (p.k_slots & 1))))
    p.k_slots--;
  p.n_cta = device_sm_count();
  p.idesc = make_idesc(128, p.NR);
  smem = TcSmem(D, p.NR, p.k_slots).bytes;
  ws = 0;
  pairs = 0;
  if (one) return p;
  pairs = (int)(((int64_t)max_rows + 2 * p.tokens - 1) / (2 * p.tokens));
  p.cap4 = ((int64_t)cap + 3) & ~(int64_t)3;
  const size_t per = (size_t)L * n_req * H * 2 * p.cap4 * sizeof(float);
  p.n_rg = (int)std::min<size_t>(pairs, std::max<size_t>(8, kTcPartBytes / per));
  p.cum = reinterpret_cast<int64_t *>(base);
  ws = ((size_t)n_req * (p.n_rg + 1) * 8 + 15) & ~size_t(15);
  p.part = reinterpret_cast<float *>(base + ws);
  ws += per * p.n_rg;
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
  int pairs;
  size_t smem, ws_bytes;
  MassTc p = tc_plan(a.n_req, a.cap, a.max_rows, a.L, a.H, a.G, D, pairs, smem, ws_bytes,
                     reinterpret_cast<uint8_t *>(ws));
  auto *kern = pairs == 0 ? k_mass_tc<D, 1> : k_mass_tc<D, 2>;
  CUtensorMap tm_k{}, tm_q{};
  p.box = a.BS % 32 == 0 ? 32 : a.BS % 16 == 0 ? 16 : a.BS % 8 == 0 ? 8 : 0;
  if ((int64_t)a.L * a.n_slots > INT32_MAX) p.box = 0;  // (a map coordinate is an int32)
  p.q_box = !a.row_idx && (int64_t)a.L * a.n_q + a.n_rows + 2 * p.tokens <= INT32_MAX;
  if (p.box && !pool_map(&tm_k, a.kpool, (int64_t)a.L * a.n_slots, a.H, D, p.box))
    return cudaErrorUnknown;
  if (p.q_box && !q_map(&tm_q, a.q, (int64_t)a.L * a.n_q, a.Hq, D, a.G, p.tokens))
    return cudaErrorUnknown;
  // (the limit is the process's: the largest, so that no thread's call lowers it
  // under another's launch)
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmemMax);
  if (e != cudaSuccess) return e;
  static std::atomic<int> regs[2];  // a thread's registers at launch (RT 1, RT 2)
  if (!regs[pairs != 0].load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa{};
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    regs[pairs != 0].store(fa.numRegs, std::memory_order_relaxed);
  }
  // setmaxnreg.inc draws on what the block was launched with
  if (regs[pairs != 0].load(std::memory_order_relaxed) * kTcThreads <
      kTcEpi * 32 * kTcMore + (kTcThreads - kTcEpi * 32) * kTcLess)
    return cudaErrorLaunchOutOfResources;
  if (pairs == 0) {
    kern<<<p.n_cta, kTcThreads, smem, s>>>(tm_k, tm_q, a, p);
    return cudaGetLastError();
  }
  const int64_t units = (int64_t)a.L * a.n_req * a.H;
  const int y = (int)std::min<int64_t>(units, 32768);
  for (p.rg0 = 0; p.rg0 < pairs && e == cudaSuccess; p.rg0 += p.n_rg) {
    k_mass_plan<<<a.n_req, 256, 0, s>>>(a, p);
    e = cudaGetLastError();
    if (e == cudaSuccess)
      e = launch_dependent(kern, dim3(p.n_cta), kTcThreads, smem, s, tm_k, tm_q, a, p);
    if (e == cudaSuccess)
      e = launch_dependent(k_mass_join,
                           dim3((a.cap + kTcKeys - 1) / kTcKeys, y, (unsigned)((units + y - 1) / y)), 256, 0, s,
                           a, p);
  }
  return e;
}

}  // namespace

size_t attn_mass_ws_bytes(int n_req, int max_blocks, int max_rows, int L, int H, int Hq, int D,
                          int BS) {
  if ((int64_t)max_rows * (Hq / H) <= kMrMaxRows) return 0;
  int pairs;
  size_t smem, ws;
  tc_plan(n_req, max_blocks * BS, max_rows, L, H, Hq / H, D, pairs, smem, ws, nullptr);
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
                       : launch_rows<128, 4>(a, s);
    return R <= 8    ? launch_rows<64, 1>(a, s)
           : R <= 16 ? launch_rows<64, 2>(a, s)
                     : launch_rows<64, 4>(a, s);
  }
  return D == 128 ? launch_tc<128>(a, ws, s) : launch_tc<64>(a, ws, s);
}

}  // namespace kvc
