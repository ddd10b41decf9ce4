// prompt_attn.cu — causal attention of the new rows of packed prompts over a
// paged cache that already holds their keys and values, one layer.  Row i of
// request r sees the positions 0 … c + i:
//   z_p = scale·q·k_p,  lse = ln Σ_p exp z_p,  out = Σ_p exp(z_p − lse)·v_p
//
// The rows of a KV head are (token, head of the group) pairs, token by token: a
// tile of up to 128 of them shares its keys whatever the group's size, and is
// causal in steps of a group.  (Groups of more than 128 heads are cut into equal
// pieces of one token.)  A unit of work is a pair of neighbouring row tiles of one
// KV head; keys pass in tiles of 128, and a unit ends with the last one its last
// row sees.
//
// k_prompt_tc, per row tile X and key tile t:
//   S_X = Q_X·Kᵀ  (M 128 rows, N 128 keys, K D; both K-major in shared memory)
//   O_X += P_X·V  (M 128 rows, N D, K 128 keys; P in tensor memory, V as it lies
//                  in the pool, MN-major)
// A softmax warpgroup per row tile, a thread per row: no exchange between threads.
// The exponent's reference is not the running maximum but the row's maximum over
// its first tile, raised only when a tile's weights sum to more than 2^30 (the sum
// is needed anyway, so the loop takes no maximum): weights, sums and O stay far
// inside fp32's and bf16's range, and the result does not depend on the reference.
// The weights stay in registers until their sum has been looked at, so that a
// tile can be worked out again on a raised reference from the S that is still there;
// they then replace S.  A raised reference rescales O in tensor memory.
//
// One warp issues the products in the order S_A(0) S_B(0) | O_A(t) S_A(t+1) O_B(t)
// S_B(t+1) | …: while one tile's weights are worked out the tensor core has the other
// tile's two products.  Four warps load, 32 keys of a tile each: TMA boxes of whole
// page rows, or cp.async row by row where a page size has no box, at the end, and for
// the values that some row of the pair does not see.
//
// Bound by the tensor core and by what hangs on its results: a pair of row tiles and 128
// keys are 32 products of 64 cycles, and S(t + 1) waits for the end of the product that
// reads P.  8192 tokens of 8 KV and 32 query heads, D 128: 414 to 418 us, 1.32 PFLOP/s, 69
// % of a library product's burst rate; 2048 behind 131072 3215 to 3250 us, 1.35 PFLOP/s.
// Without any softmax the latter would take 2960, without the loads too no less: so neither
// is what a step is spent on.  An issuer per row tile lets the two fall into step (3758 us), the
// weights handed over 64 keys at a time cost 3380, two threads a row 3247.
#include <float.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "tree_rows.cuh"

namespace kvc {
namespace {

constexpr int kPaKeys = 128;
constexpr int kPaThreads = 512;
// Registers of a softmax thread, of the others: 256·176 + 256·80 is the launch's 512·128.
constexpr int kPaMore = 176, kPaLess = 80;
constexpr float kPaUnset = -FLT_MAX;      // reference of a row that has seen nothing
constexpr float kPaMost = 1073741824.f;   // 2^30: sum of a tile's weights that raises the reference
constexpr float kPaRound = 1048576.f;     // |reference| from which logits are rounded before the difference
constexpr int kPaSlots = 8;               // ring slots, at most

struct PromptTc {
  int box;              // rows of a TMA box (a divisor of the page size), 0: no TMA
  int gc, n_ch;         // heads of a row tile's piece of the group, pieces
  int tpt;              // tokens of a row tile
  int NS;               // ring slots
  int wide;             // out is aligned to 32 bytes
  uint32_t idesc_s, idesc_o;
};

struct PromptHead {
  uint64_t full[kPaSlots], empty[kPaSlots];  // ring slots
  uint64_t qfull, sfull[2], pready[2], pvdone[2];
  uint32_t tmem_holder;
  volatile int failed, odd, bad;
};
constexpr uint32_t kPaHead = 1024;
static_assert(sizeof(PromptHead) <= kPaHead, "the head's room");

// K-major operand with the 128-byte swizzle, atoms of eight rows `sbo` bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(sbo >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major: 64 MN elements by 8 K rows an atom, atoms along K `sbo` apart, along MN `lbo`.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(sbo >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// tcgen05.mma with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(x));
  return x != 0;
}
__device__ __forceinline__ void tma_load_5d_if(uint32_t lead, uint32_t dst, const CUtensorMap *map, int x,
                                               int y, int z, int w, int v, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %8, 0;\n"
      " @q cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar), "r"(lead)
      : "memory");
}
// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_put32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 32 bytes, a whole sector (dst aligned to 32 bytes).
__device__ __forceinline__ void st_global32(void *dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void tmem_put_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Pairs of row tiles of request r (0: nothing to do).
__device__ __forceinline__ int prompt_pairs(const TreeArgs &a, const PromptTc &p, int r) {
  int c, q0, T;
  if (!tree_request(a, r, c, q0, T)) return 0;
  return ((T + p.tpt - 1) / p.tpt * p.n_ch + 1) / 2;
}

// CL: a cluster shares a unit, each CTA a part of its keys, and joins the parts from one
// another's shared memory.
template <int D, bool CL>
__global__ void __launch_bounds__(kPaThreads, 1)
k_prompt_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
            const __grid_constant__ CUtensorMap tm_q, TreeArgs a, PromptTc p) {
  constexpr int CH = D / 8, KB = D / 64;
  constexpr uint32_t kSlot = kPaKeys * D * 2, kQTile = 128 * D * 2, kAtoms = 1024 * KB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PromptHead &sm = *reinterpret_cast<PromptHead *>(base);
  const uint32_t q_u = smem_u32(base) + kPaHead, ring_u = q_u + 2 * kQTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (blockIdx.x == 0)  // one report per bad request
    for (int r = tid; r < a.n_req; r += kPaThreads) {
      int c, q0, T;
      if (!tree_request(a, r, c, q0, T)) record_error(a.status, KVC_ERR_BOUNDS);
    }
  // this CTA's unit: requests in order, a request's last rows first (they see the most)
  auto units = [&](int r) { return (int64_t)a.H * prompt_pairs(a, p, r); };
  const WarpSums sums = warp_sums(a.n_req, units);
  const int S = CL ? (int)cluster_nrank() : 1, rank = CL ? (int)cluster_rank() : 0;
  const int64_t unit = CL ? blockIdx.x / S : blockIdx.x;
  if (unit >= sums.total) return;  // (the whole cluster)
  int r, c, q0, T;
  int64_t before;
  warp_find(sums, a.n_req, unit, units, r, before);
  tree_request(a, r, c, q0, T);
  const int at = (int)(unit - before), h = at % a.H;
  const int pair = prompt_pairs(a, p, r) - 1 - at / a.H;
  // row tile x of the pair: pieces of the group inside, tokens outside
  const int n_tiles = (T + p.tpt - 1) / p.tpt * p.n_ch;
  auto token_of = [&](int x) { return (2 * pair + x) / p.n_ch * p.tpt; };
  auto piece_of = [&](int x) { return (2 * pair + x) % p.n_ch; };
  auto tiles_of = [&](int x) {  // key tiles that some row of row tile x sees
    return 2 * pair + x < n_tiles ? (c + min(T, token_of(x) + p.tpt) + kPaKeys - 1) / kPaKeys : 0;
  };
  const int tok0 = token_of(0);
  const int end = c + min(T, token_of(tiles_of(1) ? 1 : 0) + p.tpt);  // positions some row sees
  // this CTA's key tiles: from t0 on, nA of them for row tile A and nB for B
  const int all = max(tiles_of(0), tiles_of(1)), t0 = all * rank / S, t1 = all * (rank + 1) / S;
  const int nA = max(min(tiles_of(0), t1) - t0, 0), nB = max(min(tiles_of(1), t1) - t0, 0), nT = max(nA, nB);

  if (tid == 0) {
    sm.failed = sm.odd = sm.bad = 0;
    for (int i = 0; i < p.NS; i++) {
      mbar_init(smem_u32(sm.full + i), 4);
      mbar_init(smem_u32(sm.empty + i), 1);
    }
    mbar_init(smem_u32(&sm.qfull), 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(smem_u32(sm.sfull + i), 1);
      mbar_init(smem_u32(sm.pready + i), 4);
      mbar_init(smem_u32(sm.pvdone + i), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) alloc_tmem_cols(&sm.tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_holder;  // S_A (P_A in its first half), S_B, O_A, O_B

  bool ok = true;
  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPaLess));
    // ------------------------------------------------------- producers
    const int key0 = (warp & 3) * 32;  // this warp's keys of a tile
    const int64_t n_blocks = a.n_slots / a.BS;
    const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
    constexpr int RPI = 32 / CH;
    const int col = lane % CH;
    if (warp == 8 && lane == 0 && nT > 0) {
      const uint32_t bar = smem_u32(&sm.qfull);
      const int n = 2 * pair + 1 < n_tiles ? 2 : 1;
      mbar_expect_tx(bar, n * p.tpt * p.gc * D * 2);
      for (int x = 0; x < n; x++)
#pragma unroll
        for (int kb = 0; kb < KB; kb++)
          tma_load_3d(q_u + x * kQTile + kb * (128 * 128), &tm_q, kb * 64,
                      h * a.G + piece_of(x) * p.gc, q0 + token_of(x), bar);
    }
    __syncwarp();
    // stages copied by cp.async and not yet handed over: up to two
    uint32_t pend0 = 0, pend1 = 0;
    auto hand_over = [&](uint32_t bar) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto flush = [&]() {
      if (!pend0) return;
      cp_wait<0>();
      hand_over(pend0);
      if (pend1) hand_over(pend1);
      pend0 = pend1 = 0;
    };
    int32_t blk, slot = -1;  // block id of the next tile's key, slot of this tile's
    auto fetch = [&](int t) {
      const int pp = (t0 + t) * kPaKeys + key0 + lane;
      blk = pp < end && t < nT ? bt[page_of(pp, a.bs_inv)] : 0;
    };
    fetch(0);
    uint32_t st = 0, round = 0;  // ring slot, times around
    for (int i = 0; i < 2 * nT && ok; i++) {
      const int t = i >> 1;
      const bool is_v = i & 1;
      const int pp = (t0 + t) * kPaKeys + key0 + lane;
      if (!is_v) {
        slot = -1;
        if (pp < end) {
          if (blk >= 0 && blk < n_blocks) {
            slot = blk * a.BS + pp - page_of(pp, a.bs_inv) * a.BS;
          } else {
            sm.bad = 1;  // (read by the softmax warps after this stage's product)
            record_error(a.status, KVC_ERR_BOUNDS);
          }
        }
        fetch(t + 1);
      }
      if (round > 0) {  // a full ring is waited for only after everything in flight is handed over
        const uint32_t bar = smem_u32(sm.empty + st), parity = (round & 1) ^ 1;
        if (!mbar_try(bar, parity)) {
          flush();
          if (!(ok = mbar_wait_bounded(bar, parity, &sm.failed))) break;
        }
      }
      const uint32_t dst = ring_u + st * kSlot + (key0 >> 3) * kAtoms;
      const uint32_t bar = smem_u32(sm.full + st);
      if (++st == (uint32_t)p.NS) st = 0, round++;
      // values past the first row's own position are looked at (below): not by TMA
      const bool hidden = is_v && (t0 + t + 1) * kPaKeys > c + tok0 + 1;
      if (p.box > 0 && !hidden && __all_sync(0xFFFFFFFFu, slot >= 0)) {
        if (lane == 0) mbar_expect_tx(bar, kSlot / 4);
        __syncwarp();
        const uint32_t ubar = uniform32(bar), udst = uniform32(dst), uh = uniform32(h);
        const CUtensorMap *tm = is_v ? &tm_v : &tm_k;
        for (int k = 0; k < 32; k += p.box) {
          const uint32_t sl = __shfl_sync(0xFFFFFFFFu, slot, k);
          tma_load_5d_if(lane == 0, udst + (k >> 3) * kAtoms, tm, 0, 0, 0, uh, sl >> 3, ubar);
        }
        continue;
      }
      const uint16_t *pool = is_v ? a.vpool : a.kpool;
      auto place = [&](int row) {
        return dst + (row >> 3) * kAtoms + (col >> 3) * 1024 + (row & 7) * 128 + (((col & 7) ^ (row & 7)) << 4);
      };
#pragma unroll 4
      for (int k = 0; k < 32 / RPI; k++) {
        const int row = k * RPI + lane / CH;
        const int32_t sl = __shfl_sync(0xFFFFFFFFu, slot, row);
        cp_async16(place(row), pool + ((int64_t)max(sl, 0) * a.H + h) * D + col * 8, sl >= 0);
      }
      cp_commit();
      if (!hidden) {
        if (!pend0) {
          pend0 = bar;
        } else if (!pend1) {
          pend1 = bar;
        } else {
          cp_wait<2>();
          hand_over(pend0);
          pend0 = pend1;
          pend1 = bar;
        }
        continue;
      }
      // A later token's V may hold infinities or NaN that some rows do not see: the product
      // gets zeros in their place, and the unit's end adds them to the rows that do.  Each
      // thread looks at what it copied, before the stage is handed over.
      flush();
      cp_wait<0>();
      bool odd = false;
#pragma unroll 1
      for (int k = 0; k < 32 / RPI; k++) {
        const int row = k * RPI + lane / CH;
        const uint32_t ad = place(row);
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
        // (what every row of the pair sees stays)
        if (mine && (t0 + t) * kPaKeys + key0 + row > c + tok0) {
          odd = true;
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(ad), "r"(w[0]), "r"(w[1]),
                       "r"(w[2]), "r"(w[3])
                       : "memory");
        }
      }
      if (odd) sm.odd = 1;
      hand_over(bar);
    }
    flush();
    cp_wait<0>();
    if (!ok) sm.failed = 1;
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPaLess));
    if (warp == 12) {
      // ------------------------------------------------------- MMA issuer
      // The whole warp runs the loop, and the lane that elect.sync names issues: the compiler
      // then knows that one thread runs and keeps the descriptors in uniform registers.  (64
      // cycles a product at N = 128; enabled by a predicate of the whole warp, 67 to 105.)
      uint32_t st = 0, round = 0;  // next stage to be waited for
      uint32_t ks = 0, vs = 0;     // slots of the K and the V tile in use
      auto stage = [&](uint32_t &slot) {
        ok = mbar_wait_bounded(smem_u32(sm.full + st), round & 1, &sm.failed);
        slot = st;
        if (++st == (uint32_t)p.NS) st = 0, round++;
      };
      auto product_s = [&](int x) {
        const uint64_t qd = desc_k(q_u + x * kQTile, 1024), kd = desc_k(ring_u + ks * kSlot, kAtoms);
        const uint32_t dst = tmem + x * 128;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4 * KB; kk++)
            mma_bf16(dst, qd + (kk >> 2) * (128 * 8) + (kk & 3) * 2,
                     kd + (kk >> 2) * (1024 / 16) + (kk & 3) * 2, p.idesc_s, kk > 0);
          mma_commit(smem_u32(sm.sfull + x));
        }
        __syncwarp();
      };
      auto done = [&](uint32_t bar) {  // arrives when everything issued so far is done
        if (elect_one()) mma_commit(bar);
        __syncwarp();
      };
      if (nT > 0) ok = mbar_wait_bounded(smem_u32(&sm.qfull), 0, &sm.failed);
      if (ok && nT > 0) stage(ks);
      if (ok && nT > 0) {
        tc_fence_after();
        if (nA) product_s(0);
        if (nB) product_s(1);
        done(smem_u32(sm.empty + ks));
      }
      for (int t = 0; t < nT && ok; t++) {
        stage(vs);
        for (int x = 0; x < 2 && ok; x++) {
          const int n = x ? nB : nA;
          if (t >= n) continue;
          ok = mbar_wait_bounded(smem_u32(sm.pready + x), t & 1, &sm.failed);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = desc_mn(ring_u + vs * kSlot, 1024, kAtoms);
          const uint32_t dst = tmem + 256 + x * 128, src = tmem + x * 128;
          const bool last = x == 1 || t >= nB;  // no other row tile takes this key tile
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kPaKeys / 16; kk++)
              mma_ts(dst, src + kk * 8, vd + kk * (2 * kAtoms / 16), p.idesc_o, t > 0 || kk > 0);
            mma_commit(smem_u32(sm.pvdone + x));
            if (last) mma_commit(smem_u32(sm.empty + vs));
          }
          __syncwarp();
          if (t + 1 < n) {
            // (the next K tile is waited for by the first row tile that takes it)
            if (x == 0 || t + 1 >= nA) stage(ks);
            if (!ok) break;
            // S takes the place of P, which the product just issued reads
            ok = mbar_wait_bounded(smem_u32(sm.pvdone + x), t & 1, &sm.failed);
            if (!ok) break;
            tc_fence_after();
            product_s(x);
            if (x == 1 || t + 1 >= nB) done(smem_u32(sm.empty + ks));
          }
        }
      }
      if (!ok) sm.failed = 1;
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPaMore));
    // --------------------------------------------------------- softmax
    const int x = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t ts = tmem + x * 128 + lanes, to = tmem + 256 + x * 128 + lanes;
    const int n = x ? nB : nA;
    const int tx = token_of(x), token = tx + row / p.gc, head = piece_of(x) * p.gc + row % p.gc;
    const bool active = 2 * pair + x < n_tiles && row < p.tpt * p.gc && token < T && head < a.G;
    const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
    const int64_t n_blocks = a.n_slots / a.BS;
    const float zs = a.zscale, hidden = zs < 0.f ? INFINITY : -INFINITY;  // −inf once scaled
    float nref = -kPaUnset, l = 0.f;
    bool rounded = false;  // (warp-uniform) some reference is so large that differences need care
    for (int t = 0; t < n && ok; t++) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.sfull + x), t & 1, &sm.failed));
      if (!ok) break;
      tc_fence_after();
      // which keys this row sees, where it is not all of them
      const bool masked = (t0 + t + 1) * kPaKeys > c + tx + 1 || __any_sync(0xFFFFFFFFu, sm.bad);
      uint32_t see[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
      if (masked) {
        const int lim = c + token + 1 - (t0 + t) * kPaKeys;
#pragma unroll
        for (int w = 0; w < 4; w++) {
          const int pp = (t0 + t) * kPaKeys + 32 * w + lane;
          bool valid = pp < end;
          if (valid) {
            const int32_t b = bt[page_of(pp, a.bs_inv)];
            valid = b >= 0 && b < n_blocks;
          }
          const int m = min(max(lim - 32 * w, 0), 32);
          see[w] = __ballot_sync(0xFFFFFFFFu, valid) & (m == 32 ? 0xFFFFFFFFu : (1u << m) - 1u);
        }
      }
      auto hide = [&](uint32_t (&z)[32], uint32_t bits) {
#pragma unroll
        for (int e = 0; e < 32; e++)
          if (!((bits >> e) & 1u)) z[e] = __float_as_uint(hidden);
      };
      // The references first: before the first tile, where weights came out too large, and
      // for every tile while they are large.
      auto raise = [&]() {
        float mx = -INFINITY;
#pragma unroll 1
        for (int w = 0; w < 4; w++) {
          uint32_t z[32];
          tmem_issue32(ts + 32 * w, z);
          tmem_wait32(z);
          const uint32_t bits = w < 2 ? (w ? see[1] : see[0]) : (w > 2 ? see[3] : see[2]);
          if (masked) hide(z, bits);
#pragma unroll
          for (int e = 0; e < 32; e++) mx = fmaxf(mx, __fmul_rn(__uint_as_float(z[e]), zs));
        }
        const float was = -nref, now = fmaxf(was, mx);
        const float f = ex2(was - now);
        if (t > 0 && __any_sync(0xFFFFFFFFu, active && f != 1.f)) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.pvdone + x), (t - 1) & 1, &sm.failed));
          if (!ok) return;
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t v[32];
            tmem_issue32(to + cc, v);
            tmem_wait32(v);
#pragma unroll
            for (int e = 0; e < 32; e++) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
            tmem_put32(to + cc, v);
            tmem_put_wait();
          }
        }
        l *= f;
        nref = -now;
        rounded = __any_sync(0xFFFFFFFFu, active && now != kPaUnset && !(fabsf(now) < kPaRound));
      };
      uint32_t pk[64];
      float sum;
      // The weights on the references at hand and their sum.  `General`: keys may be hidden,
      // and after a raise the largest rounded product is the reference, so the difference is
      // taken from rounded products and is at most 0, however large they are.
      auto weights = [&](auto General, bool raised) {
        const uint64_t zs2 = pk2(zs, zs), nr2 = pk2(nref, nref);
        uint64_t s2[2] = {0, 0};
        uint32_t z[2][32];
        tmem_issue32(ts, z[0]);
#pragma unroll
        for (int w = 0; w < 4; w++) {
          tmem_wait32(z[w & 1]);
          if (w < 3) tmem_issue32(ts + 32 * (w + 1), z[(w + 1) & 1]);
          if (General.value && masked) hide(z[w & 1], see[w]);
#pragma unroll
          for (int e = 0; e < 16; e++) {
            float u = __uint_as_float(z[w & 1][2 * e]), v = __uint_as_float(z[w & 1][2 * e + 1]);
            if (General.value && raised) {
              u = __fadd_rn(__fmul_rn(u, zs), nref);
              v = __fadd_rn(__fmul_rn(v, zs), nref);
            } else {
              upk2(fma2(pk2(u, v), zs2, nr2), u, v);
            }
            u = ex2(u);
            v = ex2(v);
            s2[e & 1] = add2(s2[e & 1], pk2(u, v));
            pk[16 * w + e] = pack_bf16x2(u, v);
          }
        }
        float u, v;
        upk2(add2(s2[0], s2[1]), u, v);
        sum = u + v;
        return __all_sync(0xFFFFFFFFu, !active || sum <= kPaMost);
      };
      bool fine = false;
      if (t > 0 && !rounded) {
        if (masked) fine = weights(std::true_type(), false);
        else fine = weights(std::false_type(), false);
      }
      if (!fine) {
        raise();
        if (!ok) break;
        weights(std::true_type(), true);
      }
      l += sum;
      tmem_put32(ts, pk);
      tmem_put32(ts + 32, pk + 32);
      tmem_put_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(sm.pready + x));
    }
    // ---- the unit's result
    if (ok && n > 0) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(sm.pvdone + x), (n - 1) & 1, &sm.failed));
      tc_fence_after();
    }
    if (CL) named_sync(1, 256);  // both row tiles' products are done: the ring takes O
    if (ok && (CL || n > 0)) {
      const float inv = CL ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const bool none = n == 0 || l == 0.f;
      const int64_t qr = (int64_t)(q0 + token) * a.Hq + h * a.G + head;
      const bool odd = sm.odd != 0;
      float4 *part = reinterpret_cast<float4 *>(base + (ring_u - smem_u32(base))) + (x * 128 + row) * (D / 4);
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 32) {
        float v[32];
        if (CL && n == 0) {
#pragma unroll
          for (int e = 0; e < 32; e++) v[e] = 0.f;
        } else {
          uint32_t z[32];
          tmem_issue32(to + cc, z);
          tmem_wait32(z);
#pragma unroll
          for (int e = 0; e < 32; e++) v[e] = none ? 0.f : __uint_as_float(z[e]) * inv;
        }
        if (odd && active) {  // infinities and NaN of later tokens, among this CTA's keys, that the row sees
          const int last = min(c + token, (t0 + nT) * kPaKeys - 1);
#pragma unroll 1
          for (int pn = max(c + tok0 + 1, t0 * kPaKeys); pn <= last; pn++) {
            const int pg = page_of(pn, a.bs_inv);
            const int32_t b = bt[pg];
            if (b < 0 || b >= n_blocks) continue;
            const uint16_t *vr = a.vpool + (((int64_t)b * a.BS + pn - pg * a.BS) * a.H + h) * D + cc;
#pragma unroll
            for (int e = 0; e < 32; e++) {
              const float vn = bf16_lo(vr[e]);
              if (!(fabsf(vn) < INFINITY)) v[e] += vn;
            }
          }
        }
        if (CL) {
          // (16-byte pieces, turned by the row so that a warp's rows lie in distinct banks)
#pragma unroll
          for (int e = 0; e < 8; e++)
            part[(cc / 4 + e) ^ (row & 7)] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else if (active) {
          uint16_t *dst = a.out + qr * D + cc;
#pragma unroll
          for (int e = 0; e < 2; e++) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; k++) w[k] = pack_bf16x2(v[16 * e + 2 * k], v[16 * e + 2 * k + 1]);
            if (p.wide) {
              st_global32(dst + 16 * e, w);
            } else {
              *reinterpret_cast<uint4 *>(dst + 16 * e) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4 *>(dst + 16 * e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      // (per row of the part, the reference and the sum, in Q's place)
      if (CL) reinterpret_cast<float2 *>(base + kPaHead)[x * 128 + row] = make_float2(none ? -INFINITY : -nref, none ? 0.f : l);
      else if (active) a.lse[qr] = l == 0.f ? -INFINITY : (log2f(l) - nref) * kLn2;
    }
    if (!ok) {
      sm.failed = 1;
      if (lane == 0) record_error(a.status, KVC_ERR_TIMEOUT);
    }
  }

  if constexpr (CL) {
    // The unit's parts are in the cluster's CTAs: added up in order, the rows dealt out to all.
    __syncwarp();
    cluster_sync_all();
    const uint32_t ml_at = q_u;
    for (int e = rank * kPaThreads + tid; e < 256 * (D / 4); e += S * kPaThreads) {
      const int xr = e / (D / 4), d4 = e % (D / 4), x = xr >> 7, row = xr & 127;
      const int token = token_of(x) + row / p.gc, head = piece_of(x) * p.gc + row % p.gc;
      if (2 * pair + x >= n_tiles || row >= p.tpt * p.gc || token >= T || head >= a.G) continue;
      float mx = -INFINITY;
      for (int k = 0; k < S; k++) mx = fmaxf(mx, ld_cluster_f2(mapa_u32(ml_at + xr * 8, k)).x);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < S; k++) {
        const float2 ml = ld_cluster_f2(mapa_u32(ml_at + xr * 8, k));
        // (a part that saw nothing of the row may still hold what is not finite)
        const float4 v = ld_cluster_f4(mapa_u32(ring_u + (xr * (D / 4) + (d4 ^ (row & 7))) * 16, k));
        const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - mx);
        sum = fmaf(ml.y, ml.x == -INFINITY ? 0.f : f, sum);
        acc.x = fmaf(v.x, share_of(v.x, f), acc.x);
        acc.y = fmaf(v.y, share_of(v.y, f), acc.y);
        acc.z = fmaf(v.z, share_of(v.z, f), acc.z);
        acc.w = fmaf(v.w, share_of(v.w, f), acc.w);
      }
      const int64_t qr = (int64_t)(q0 + token) * a.Hq + h * a.G + head;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint2 *>(a.out + qr * D + 4 * d4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (d4 == 0) a.lse[qr] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
    __syncwarp();
    cluster_sync_all();  // (no CTA leaves while another reads its part)
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
    mbar_drain(smem_u32(&sm.qfull), 0);
    for (int i = 0; i < 2; i++) {
      mbar_drain(smem_u32(sm.sfull + i), 0);
      mbar_drain(smem_u32(sm.sfull + i), 1);
      mbar_drain(smem_u32(sm.pvdone + i), 0);
      mbar_drain(smem_u32(sm.pvdone + i), 1);
    }
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    free_tmem_cols(tmem, 512);
  }
}

// Boxes of `box` consecutive slots (a multiple of 8) of one head, both halves of a row of
// 128 elements: [group of 8 slots][half][slot][64 columns], 128-byte swizzle.
bool rows_map(CUtensorMap *m, const void *pool, int64_t n_slots, int H, int D, int box) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t row = (cuuint64_t)H * D * 2;
  cuuint64_t dims[5] = {64, 8, (cuuint64_t)D / 64, (cuuint64_t)H, (cuuint64_t)n_slots / 8};
  cuuint64_t strides[4] = {row, 128, (cuuint64_t)D * 2, 8 * row};
  cuuint32_t bx[5] = {64, 8, (cuuint32_t)D / 64, 1, (cuuint32_t)box / 8}, es[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(pool), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs that share a unit (1, 2, 4 or 8), in key tiles that a CTA takes one after another:
// waves of CTAs, each with its share of a unit's keys, a beginning and an end worth about
// four tiles, and the join's two.  An SM holds one CTA, and clusters of 4 and 8 leave
// some SMs of a GPC empty.  8 KV and 32 query heads, D 128, in us by 1, 2, 4 and 8: 17
// rows behind 8192 95, 60, 36, 25; 256 behind 65536 792, 422, 222, 351; 512 (twice) behind
// 16384 213, 245, 272, 380; a prompt of 300 14, 21, 20, 21; of 1024 23, 43, 71, 154.
// The keys are the table's width, for the lengths lie on the device; these figures are of
// tables as long as the requests.  In wide ones a short prompt may go to a cluster: 300 rows,
// a call alone after an L2 flush, 20 us in an exact table, 26 in one of 8K, 58 in one of 32K.
int prompt_cluster(int64_t units, int64_t kt) {
  const double sms = device_sm_count();
  int best = 1;
  double least = 0;
  for (int S = 1; S <= 8 && S <= kt; S *= 2) {
    const double room = S == 8 ? 0.84 * sms : S == 4 ? 0.94 * sms : sms;
    const double cost = ceil(units * S / room) * (ceil((double)kt / S) + (S > 1 ? 6 : 4));
    if (S == 1 || cost < least) {
      least = cost;
      best = S;
    }
  }
  return best;
}

template <int D>
cudaError_t launch_prompt_tc(const TreeArgs &a, int max_rows, cudaStream_t s) {
  constexpr size_t kSmemMax = 232448;
  constexpr size_t kSlot = kPaKeys * D * 2, kFixed = 1024 + kPaHead + 2 * 128 * D * 2;
  static_assert(kFixed + 4 * kSlot <= kSmemMax && 4 * kSlot >= 256 * D * 4, "the parts' O fit the ring");
  PromptTc p{};
  p.n_ch = (a.G + 127) / 128;
  p.gc = (a.G + p.n_ch - 1) / p.n_ch;
  p.tpt = 128 / p.gc;
  p.NS = (int)std::min<size_t>(kPaSlots, (kSmemMax - kFixed) / kSlot);
  // (8192 tokens, a call alone after an L2 flush: pages of 64 to 16 408 us, of 8 411; of 12, row
  // by row, 469)
  p.box = a.BS % 32 == 0 ? 32 : a.BS % 16 == 0 ? 16 : a.BS % 8 == 0 ? 8 : 0;
  p.wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  p.idesc_s = make_idesc(128, kPaKeys);
  p.idesc_o = make_idesc(128, D) | (1u << 16);  // B (V) MN-major
  CUtensorMap tm_k{}, tm_v{}, tm_q{};
  if (p.box && !(rows_map(&tm_k, a.kpool, a.n_slots, a.H, D, p.box) &&
                 rows_map(&tm_v, a.vpool, a.n_slots, a.H, D, p.box)))
    return cudaErrorUnknown;
  if (!q_map(&tm_q, a.q, a.n_q, a.Hq, D, p.gc, p.tpt)) return cudaErrorUnknown;
  // units at most: every request's last pair may be part empty
  const int64_t each = ((int64_t)(max_rows + p.tpt - 1) / p.tpt * p.n_ch + 1) / 2;
  const int64_t rows = std::min<int64_t>(a.n_q, (int64_t)a.n_req * max_rows);
  const int64_t pairs = std::min<int64_t>(a.n_req * each, rows * p.n_ch / (2 * p.tpt) + 2 * (int64_t)a.n_req);
  const int64_t units = pairs * a.H;
  const int S = prompt_cluster(units, ((int64_t)a.max_blocks * a.BS + kPaKeys - 1) / kPaKeys);
  if (units * S > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto *kern = S > 1 ? k_prompt_tc<D, true> : k_prompt_tc<D, false>;
  // (the limit is the process's: the largest, so that no thread's call lowers it under
  // another's launch)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
  if (e != cudaSuccess) return e;
  static std::atomic<int> known[2];  // a thread's registers at launch
  std::atomic<int> &regs = known[S > 1];
  if (!regs.load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa{};
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  // setmaxnreg.inc draws on what the block was launched with
  if (regs.load(std::memory_order_relaxed) * kPaThreads < 256 * (kPaMore + kPaLess))
    return cudaErrorLaunchOutOfResources;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * S));
  cfg.blockDim = dim3(kPaThreads);
  cfg.dynamicSmemBytes = kFixed + p.NS * kSlot;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)S;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, tm_q, a, p);
}

}  // namespace

cudaError_t launch_prompt_attn(const uint16_t *q, const uint16_t *kpool, const uint16_t *vpool,
                               int64_t n_slots, const int32_t *block_table, int max_blocks,
                               const int32_t *ctx_len, const int32_t *q_off, int n_req, int n_q,
                               int max_rows, int H, int Hq, int D, int BS, float scale,
                               uint16_t *out, float *lse, int32_t *status, cudaStream_t s) {
  TreeArgs a{};
  a.q = q, a.kpool = kpool, a.vpool = vpool, a.block_table = block_table;
  a.ctx_len = ctx_len, a.q_off = q_off, a.out = out, a.lse = lse, a.status = status;
  a.n_slots = n_slots, a.max_blocks = max_blocks, a.n_req = n_req, a.n_q = n_q;
  a.max_tree = max_rows, a.H = H, a.Hq = Hq, a.G = Hq / H, a.BS = BS, a.bs_inv = page_inverse(BS);
  a.zscale = scale != 0.f ? scale * kLog2e : 1e-30f;  // (so that −inf stays −inf when scaled)
  return D == 128 ? launch_prompt_tc<128>(a, max_rows, s) : launch_prompt_tc<64>(a, max_rows, s);
}

}  // namespace kvc
