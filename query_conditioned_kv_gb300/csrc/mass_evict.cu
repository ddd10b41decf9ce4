// mass_evict.cu — eviction by accumulated attention weight, per (layer,
// request, KV head) segment, with the cache made dense in place.
//
// Per segment of n rows and a budget B < n: rows are ranked by (pinned,
// weight descending, lower row first) and the first B stay.  A pinned row
// (original position among the first n_sink or the last n_recent tokens)
// gets the largest key, so one exact radix selection of the B-th largest key
// gives the staying set; equal keys at the threshold stay lowest row first.
// The staying rows at or past B then fill the rows below B that leave, k-th
// to k-th.  Sources are all ≥ B and destinations all < B, so the copies need
// no order and no buffer, and their traffic is what the step evicts: at most
// min(B, n − B) rows, against up to B rows for a chronological compaction.
//
// One launch.  A cluster of S CTAs takes a segment: each stages the keys and
// selects by itself (the weights come from L2 after the first reader), rank 0
// writes the weights and positions, and the row copies are split over the
// ranks, so a few segments still use the whole GPU.  The cluster barrier
// before a leaving row's weight is overwritten lets mass_out/pos_out be
// mass/pos.  After the first radix level only the keys in its digit are looked
// at (a list in shared memory), and the levels end once all of them stay.
//
// Bound: few rows leave, latency (64 of 4160 rows, 288 segments: 16.5 us, 2.3 TB/s;
// weights, levels, sweep, block ids and rows wait for one another, about 15
// thousand cycles); many, random 256-byte pieces read and written (6K to 4K, 1152
// segments: 206 to 247 us from one block table to another, 64 to 77 % of a plain
// copy's rate; 512 threads a CTA 5 % more, eight rows in flight a warp slower than
// four).  By the table's length, 64 of 4160 rows: up to 16K positions 17 us, to 48K 25
// (one CTA of 1024 threads per SM), past the staged length 50 (weights and positions
// read again at every level, one CTA per segment).
#include <algorithm>

#include "kvc_internal.cuh"
#include "mma_ptx.cuh"
#include "radix_select.cuh"
#include "tc_ptx.cuh"

namespace kvc {
namespace {

constexpr int kEvThreads = 512;      // few segments
constexpr int kEvThreadsMany = 256;  // many: more CTAs per SM, one's copies under another's selection
constexpr int kEvThreadsBig = 1024;  // long segments
constexpr int kEvList = 1024;        // keys listed after the first level
constexpr int kEvBigFrom = 16384;    // rows past which a segment takes kEvThreadsBig

// Dynamic shared memory of a staged segment of `rows` rows.
constexpr size_t staged_bytes(int rows) {
  return ((size_t)rows + rows / 32 + 2) * sizeof(uint32_t);
}

struct EvictArgs {
  uint16_t *kpool, *vpool;  // [L][n_slots][H][D]
  const int32_t *block_table;
  const int32_t *seqused, *n_pos, *t_end;
  const float *mass;
  const int32_t *pos;
  float *mass_out;
  int32_t *pos_out, *n_out, *status;
  int32_t *lists;  // streaming segments: [n_seg][2][cap]
  int64_t n_slots;
  int n_req, H, D, BS, max_blocks, cap, budget, n_sink, n_recent;
  uint32_t bs_inv;  // page_inverse(BS)
};

struct Row {
  const float *mass;
  const int32_t *pos;
  int n, n_pos, t_end, n_sink;
  int64_t recent0;
  __device__ int origin(int i) const { return i < n_pos ? pos[i] : t_end - (n - i); }
  __device__ uint32_t key(float m, int o, bool &nan) const {
    const uint32_t k = order_key(m, nan);
    return o < n_sink || o >= recent0 ? 0xFFFFFFFFu : k;
  }
  __device__ uint32_t key(int i, bool &nan) const { return key(mass[i], origin(i), nan); }
};

template <bool STAGED, int NT>
__global__ void __launch_bounds__(NT)
k_mass_evict(EvictArgs a) {
  extern __shared__ uint32_t dyn[];  // keys [kp(cap)], then the two lists in their place
  __shared__ uint32_t hist[kSelHist * 256];
  __shared__ uint32_t warp_tot[32];
  __shared__ uint32_t s_kmax, s_kmin, s_prefix, s_need, s_have, n_list;
  __shared__ uint32_t list[STAGED ? kEvList : 1];

  const int S = (int)tc::cluster_nrank(), rank = (int)tc::cluster_rank();
  const int seg = blockIdx.x / S;
  const int h = seg % a.H, r = (seg / a.H) % a.n_req;
  const int64_t l = seg / (a.H * a.n_req);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // a thread's first rows, asked for together with the sizes (any row below cap
  // may be read); the block ids on their way to L1, and the first level's
  // histogram cleared, meanwhile.  (4, 6, 10 or 16 of them: 1100 rows 13.1, 13.3,
  // 14.0 and 14.8 us, 8 requests of 2112 56, 55, 53 and 54, 4 of 6144 265, 263, 262
  // and 260.)
  constexpr int U1 = 10;
  const int64_t base = (int64_t)seg * a.cap;
  float m[U1];
  int o[U1];
#pragma unroll
  for (int u = 0; u < U1; u++) {
    const int i = u * NT + tid;
    m[u] = i < a.cap ? a.mass[base + i] : 0.f;
    o[u] = i < a.cap ? a.pos[base + i] : 0;
  }
  const int32_t *bt = a.block_table + (int64_t)r * a.max_blocks;
  for (int i = 32 * tid; i < a.max_blocks; i += 32 * NT)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(bt + i));
  for (int j = tid; j < kSelHist * 256; j += NT) hist[j] = 0u;
  if (tid == 0) {
    s_kmax = 0u;
    s_kmin = 0xFFFFFFFFu;
  }
  __syncthreads();
  const int n = a.seqused[r], B = a.budget;
  const bool bad = n < 0 || n > a.cap;
  float *mass_out = a.mass_out + base;
  int32_t *pos_out = a.pos_out + base;
  Row row;
  row.mass = a.mass + base;
  row.pos = a.pos + base;
  row.n = n;
  row.n_pos = min(max(a.n_pos[r], 0), max(n, 0));
  row.t_end = a.t_end[r];
  row.n_sink = a.n_sink;
  row.recent0 = (int64_t)row.t_end - a.n_recent;
  if (l == 0 && h == 0 && rank == 0 && tid == 0) {
    a.n_out[r] = bad ? 0 : min(n, B);
    if (bad) record_error(a.status, KVC_ERR_BOUNDS);
  }
  if (bad || n <= B) {  // every CTA of the cluster alike
    if (rank == 0)
      for (int i = tid; i < n && !bad; i += NT) {
        mass_out[i] = row.mass[i];
        pos_out[i] = row.origin(i);
      }
    return;
  }

  uint32_t *keys = dyn;
  bool nan = false;
  uint32_t kmax = 0u, kmin = 0xFFFFFFFFu;
  // rows below B keep their place (the ones that leave are overwritten below);
  // in place, rewriting a weight changes nothing
  const bool writes = rank == 0 && (a.mass_out != a.mass || a.pos_out != a.pos || row.n_pos < B);
  for (int b0 = 0;;) {
#pragma unroll
    for (int u = 0; u < U1; u++) {
      const int i = b0 + u * NT + tid;
      if (i < n) {
        if (i >= row.n_pos) o[u] = row.t_end - (n - i);
        const uint32_t key = row.key(m[u], o[u], nan);
        if (STAGED) keys[kp(i)] = key;
        kmax = max(kmax, key);
        kmin = min(kmin, key);
        if (i < B && writes) {
          mass_out[i] = m[u];
          pos_out[i] = o[u];
        }
      }
    }
    b0 += NT * U1;
    if (b0 >= n) break;
#pragma unroll
    for (int u = 0; u < U1; u++) {
      const int i = b0 + u * NT + tid;
      m[u] = i < n ? row.mass[i] : 0.f;
      o[u] = i < row.n_pos ? row.pos[i] : 0;
    }
  }
  if (nan) record_error(a.status, KVC_ERR_NAN);
  kmax = __reduce_max_sync(0xFFFFFFFFu, kmax);
  kmin = __reduce_min_sync(0xFFFFFFFFu, kmin);
  if (lane == 0) {
    atomicMax(&s_kmax, kmax);
    atomicMin(&s_kmin, kmin);
  }
  __syncthreads();
  kmax = s_kmax;
  kmin = s_kmin;
  // the B-th largest key: eight bits per level from the highest bit in which
  // the keys differ, each level a histogram of the keys that still match
  uint32_t need = (uint32_t)B;
  int hi = kmax == kmin ? -1 : 31 - __clz(kmax ^ kmin);
  uint32_t prefix = hi < 0 ? kmax : hi == 31 ? 0u : (kmax >> (hi + 1)) << (hi + 1);
  uint32_t have = (uint32_t)n;  // keys with the prefix
  bool listed = false, clear = true;  // (the histogram is)
  while (hi >= 0 && have > need) {
    const int lo = hi >= 7 ? hi - 7 : 0;
    const uint32_t dmask = (2u << (hi - lo)) - 1u;
    const uint32_t pmask = hi == 31 ? 0u : ~((2u << hi) - 1u);
    uint32_t *hw = hist + (warp % kSelHist) * 256;
    if (!clear)
      for (int j = tid; j < kSelHist * 256; j += NT) hist[j] = 0u;
    __syncthreads();
    clear = false;
    if (listed) {
      for (int i = tid; i < (int)n_list; i += NT)
        if ((list[i] & pmask) == prefix) atomicAdd(&hw[(list[i] >> lo) & dmask], 1u);
    } else {
#pragma unroll 4
      for (int i = tid; i < n; i += NT) {
        const uint32_t key = STAGED ? keys[kp(i)] : row.key(i, nan);
        if ((key & pmask) == prefix) atomicAdd(&hw[(key >> lo) & dmask], 1u);
      }
    }
    if (tid == 0 && !listed) {
      n_list = 0;
      s_kmax = 0u;
      s_kmin = 0xFFFFFFFFu;
    }
    __syncthreads();
    if (warp == 0) pick_digit(hist, lane, prefix, need, lo, &s_prefix, &s_need, &s_have);
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    have = s_have;
    hi = lo - 1;
    if (STAGED && !listed && have <= kEvList && hi >= 0 && have > need) {
      const uint32_t next = ~((2u << hi) - 1u);  // (its order does not matter)
      uint32_t mx = 0u, mn = 0xFFFFFFFFu;
#pragma unroll 4
      for (int i = tid; i < n; i += NT) {
        const uint32_t key = keys[kp(i)];
        if ((key & next) == prefix) {
          list[atomicAdd(&n_list, 1u)] = key;
          mx = max(mx, key);
          mn = min(mn, key);
        }
      }
      // their common leading bits need no level (equal weights: none at all)
      if (mx >= mn) {
        atomicMax(&s_kmax, mx);
        atomicMin(&s_kmin, mn);
      }
      __syncthreads();
      const uint32_t diff = s_kmax ^ s_kmin;
      hi = diff ? 31 - __clz(diff) : -1;
      prefix = hi < 0 ? s_kmax : (s_kmax >> (hi + 1)) << (hi + 1);
      listed = true;
    }
  }
  // all that have the prefix stay: no row is equal to the threshold (prefix > 0,
  // for some key is lower, unless all are equal)
  const bool ties = have > need;
  const uint32_t thr = ties ? prefix : prefix - 1;
  if (!ties) need = 0;

  // Ordered sweep in rounds of up to 64 rows per thread: stay = key > thr or
  // one of the first `need` rows with key == thr.  Rows below B that leave and
  // rows past B that stay are numbered by a block scan.
  int32_t *holes = STAGED ? reinterpret_cast<int32_t *>(keys) : a.lists + 2 * base;
  int32_t *tails = holes + (STAGED ? a.cap / 2 + 1 : a.cap);
  const int ipt = STAGED ? (n + NT - 1) / NT : 64;
  uint32_t eq_carry = 0, hole_carry = 0, tail_carry = 0;
  for (int b0 = 0; b0 < n; b0 += NT * ipt) {
    const int i0 = min(n, b0 + tid * ipt), cnt = min(n, i0 + ipt) - i0;
    uint64_t eqm = 0, km = 0;
#pragma unroll 4
    for (int e = 0; e < cnt; e++) {
      const uint32_t key = STAGED ? keys[kp(i0 + e)] : row.key(i0 + e, nan);
      km |= (uint64_t)(key > thr) << e;
      eqm |= (uint64_t)(key == thr) << e;
    }
    uint32_t tot;
    if (ties) {
      const uint32_t eq_before =
          eq_carry + block_excl_scan((uint32_t)__popcll(eqm), &tot, warp_tot);
      eq_carry += tot;
      if (eq_before < need) {
        const uint32_t take = min((uint32_t)__popcll(eqm), need - eq_before);
        for (uint32_t t = 0; t < take; t++) {
          km |= eqm & (~eqm + 1);  // lowest remaining equal row
          eqm &= eqm - 1;
        }
      }
    }
    // rows of this chunk below B: bits [0, nb)
    const int nb = max(0, min(cnt, B - i0));
    const uint64_t below = nb >= 64 ? ~0ull : (1ull << nb) - 1ull;
    uint64_t hm = ~km & below, tm = km & ~below;
    uint32_t hk, tk;
    if (STAGED) {  // at most min(B, n − B) < 2^16 of each: one scan of both
      const uint32_t both = block_excl_scan(
          (uint32_t)__popcll(hm) | (uint32_t)__popcll(tm) << 16, &tot, warp_tot);
      hk = both & 0xFFFFu;
      tk = both >> 16;
      hole_carry = tot & 0xFFFFu;
      tail_carry = tot >> 16;
    } else {
      hk = hole_carry + block_excl_scan((uint32_t)__popcll(hm), &tot, warp_tot);
      hole_carry += tot;
      tk = tail_carry + block_excl_scan((uint32_t)__popcll(tm), &tot, warp_tot);
      tail_carry += tot;
    }
    // (the scans' barriers: every thread has read its keys, which the lists replace)
    for (; hm; hm &= hm - 1) holes[hk++] = i0 + __ffsll((long long)hm) - 1;
    for (; tm; tm &= tm - 1) tails[tk++] = i0 + __ffsll((long long)tm) - 1;
  }
  if (S > 1) tc::cluster_sync_all();  // every rank has read mass and pos
  else __syncthreads();
  const int n_pairs = (int)tail_carry;  // = hole_carry

  // the moved rows' weights and positions, by the threads whose rows below come last
  const int k_mine = NT - 1 - tid;
  float m_moved = 0.f;
  int o_moved = 0;
  const bool moves = rank == 0 && k_mine < n_pairs;
  if (moves) {
    m_moved = row.mass[tails[k_mine]];
    o_moved = row.origin(tails[k_mine]);
  }

  // K and V rows: 16-byte columns, a warp takes pairs in turn
  const int cols = a.D / 8;          // columns of one row: 8 or 16
  const int per = 32 / (2 * cols);   // pairs a warp moves at once (K and V together)
  const int sub = lane / (2 * cols), c2 = lane % (2 * cols);
  uint16_t *pool = (c2 < cols ? a.kpool : a.vpool) + l * a.n_slots * a.H * a.D + h * a.D +
                   (c2 % cols) * 8;
  const int64_t n_blocks = a.n_slots / a.BS, stride = (int64_t)a.H * a.D;
  const int step = (NT / 32) * S * per;
  constexpr int U = 4;
  for (int k0 = (rank * (NT / 32) + warp) * per + sub; k0 < n_pairs; k0 += step * U) {
    uint4 v[U];
    int64_t d[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int k = k0 + u * step;
      d[u] = -1;
      if (k < n_pairs) {
        const int pd = holes[k], ps = tails[k];
        const int gd = page_of(pd, a.bs_inv), gs = page_of(ps, a.bs_inv);
        const int32_t bd = bt[gd], bs = bt[gs];
        if (bd >= 0 && bd < n_blocks && bs >= 0 && bs < n_blocks) {
          d[u] = ((int64_t)bd * a.BS + pd - gd * a.BS) * stride;
          v[u] = ld_stream(pool + ((int64_t)bs * a.BS + ps - gs * a.BS) * stride);
        } else {
          record_error(a.status, KVC_ERR_BOUNDS);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++)
      if (d[u] >= 0) st_stream(pool + d[u], v[u]);
  }

  if (moves) {
    mass_out[holes[k_mine]] = m_moved;
    pos_out[holes[k_mine]] = o_moved;
  }
  if (rank == 0)
    for (int k = k_mine + NT; k < n_pairs; k += NT) {
      const int d = holes[k], s = tails[k];
      mass_out[d] = row.mass[s];
      pos_out[d] = row.origin(s);
    }
}

}  // namespace

size_t mass_evict_ws_bytes(int n_req, int max_blocks, int L, int H, int BS, int budget) {
  const int64_t cap = (int64_t)max_blocks * BS;
  if (cap <= KVC_EVICT_STAGED_ROWS) return 0;
  return (size_t)L * n_req * H * 2 * cap * sizeof(int32_t);
}

cudaError_t launch_mass_evict(uint16_t *kpool, uint16_t *vpool, int64_t n_slots,
                              const int32_t *block_table, int max_blocks,
                              const int32_t *seqused, const int32_t *n_pos,
                              const int32_t *t_end, const float *mass, const int32_t *pos,
                              float *mass_out, int32_t *pos_out, int32_t *n_out, int n_req,
                              int L, int H, int D, int BS, int budget, int n_sink, int n_recent,
                              void *ws, int32_t *status, cudaStream_t s) {
  EvictArgs a{kpool,     vpool,    block_table, seqused, n_pos,   t_end,
              mass,      pos,      mass_out,    pos_out, n_out,   status,
              reinterpret_cast<int32_t *>(ws),  n_slots, n_req,   H,
              D,         BS,       max_blocks,  max_blocks * BS,  budget,
              n_sink,    n_recent, page_inverse(BS)};
  const int n_seg = L * n_req * H;
  const bool staged = a.cap <= KVC_EVICT_STAGED_ROWS, many = n_seg >= 4 * device_sm_count();
  const int nt = a.cap > kEvBigFrom ? kEvThreadsBig : many ? kEvThreadsMany : kEvThreads;
  auto *kern = !staged               ? k_mass_evict<false, kEvThreadsBig>
               : nt == kEvThreadsBig ? k_mass_evict<true, kEvThreadsBig>
               : many                ? k_mass_evict<true, kEvThreadsMany>
                                     : k_mass_evict<true, kEvThreads>;
  size_t smem = 0;
  if (staged) {
    // the limit is the process's: the kernel's largest, so that no thread's call
    // lowers it under another's launch
    smem = staged_bytes(a.cap);
    const int most = (int)staged_bytes(nt == kEvThreadsBig ? KVC_EVICT_STAGED_ROWS : kEvBigFrom);
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  // a cluster per segment while segments are few: two CTAs per SM in all
  int S = 1;
  if (staged)
    while (S < 8 && n_seg * S * 2 <= 2 * device_sm_count()) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)n_seg * S));
  cfg.blockDim = dim3(nt);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)S;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace kvc
