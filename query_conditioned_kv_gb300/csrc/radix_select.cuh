// radix_select.cuh — building blocks of the exact radix selections (select.cu,
// mass_evict.cu): order-preserving keys, a block scan and one radix level.
#pragma once

#include "kvc_internal.cuh"

namespace kvc {
namespace {

// Histogram copies of the radix levels (warp w counts into copy w mod 8), so
// conflicting atomics come from at most a few warps.
constexpr int kSelHist = 8;

// Keys are stored with one pad word per 32: a thread's contiguous chunk and
// the strided sweeps both read distinct banks.
__device__ __forceinline__ int kp(int i) { return i + (i >> 5); }

__device__ __forceinline__ uint32_t order_key(float s, bool &nan) {
  if (s != s) {
    nan = true;
    return 0u;
  }
  if (s == 0.f) s = 0.f;  // −0.0 ranks with +0.0
  uint32_t u = __float_as_uint(s);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive block scan of v (all threads); *total gets the block sum.
__device__ __forceinline__ uint32_t block_excl_scan(uint32_t v, uint32_t *total,
                                                    uint32_t *warp_tot) {
  int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n_warps = blockDim.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t t = lane < n_warps ? warp_tot[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      uint32_t y = __shfl_up_sync(0xFFFFFFFFu, t, o);
      if (lane >= o) t += y;
    }
    warp_tot[lane] = t;
  }
  __syncthreads();
  uint32_t excl = x - v + (warp > 0 ? warp_tot[warp - 1] : 0u);
  *total = warp_tot[n_warps - 1];
  __syncthreads();
  return excl;
}

// Warp 0: from the radix level's histograms (kSelHist copies of 256 bins),
// the largest digit d whose count from the top reaches `need`; writes the
// extended prefix, the count still needed among the keys with that prefix and
// (where asked for) how many keys have it.
__device__ __forceinline__ void pick_digit(const uint32_t *hist, int lane, uint32_t prefix,
                                           uint32_t need, int lo, uint32_t *s_prefix,
                                           uint32_t *s_need, uint32_t *s_have = nullptr) {
  // lane l: bins 8l … 8l+7 summed over the histogram copies
  uint32_t loc[8], lsum = 0;
#pragma unroll
  for (int b = 0; b < 8; b++) {
    uint32_t v = 0;
    for (int c = 0; c < kSelHist; c++) v += hist[c * 256 + 8 * lane + b];
    loc[b] = v;
    lsum += v;
  }
  uint32_t sfx = lsum;  // Σ of the bins ≥ 8·lane
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_down_sync(0xFFFFFFFFu, sfx, o);
    if (lane + o < 32) sfx += y;
  }
  const uint32_t above = sfx - lsum;  // Σ of the bins ≥ 8·(lane + 1)
  if (above < need && sfx >= need) {  // exactly one lane
    uint32_t acc = above, have = 0;
    int d = 8 * lane;
#pragma unroll
    for (int b = 7; b >= 0; b--)
      if (acc + loc[b] >= need) {
        d = 8 * lane + b;
        have = loc[b];
        break;
      } else {
        acc += loc[b];
      }
    *s_prefix = prefix | ((uint32_t)d << lo);
    *s_need = need - acc;
    if (s_have) *s_have = have;
  }
}

}  // namespace
}  // namespace kvc
