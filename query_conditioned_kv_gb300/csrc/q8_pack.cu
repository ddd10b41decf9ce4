// q8_pack.cu — blocks of a paged bf16 cache in 8 bits: per (layer, block, head)
// and for K and V apart, the least power of two s whose 448-fold holds the
// block's largest value, and e4m3(x / s).
//
// A power of two loses nothing against amax / 448: e4m3 is a floating format
// whose relative step does not depend on the scale, and the division is exact.
// Bound by HBM: 2 bytes read and 1 written per value, every value once.  A
// group of one, two or four warps holds a head's block in registers between
// the maximum and the conversion (16 bytes a load, BS·D/8 of them), so that
// nothing is read twice; neighbouring heads lie in neighbouring warps, for a
// row of a page is contiguous over its heads.
#include <cuda_fp8.h>

#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr int kPackWarps = 8;
constexpr int kPackLoads = 8;  // 16-byte loads of a lane

struct Q8PackArgs {
  const uint16_t *kpool, *vpool;
  uint8_t *k8, *v8;
  float *kscale, *vscale;
  const int32_t *src, *dst;
  int32_t *status;
  int64_t n_blocks, n_blocks8;
  int H, BS, hgroups;  // CTAs of one (pair, layer, pool)
};

template <int D, int WPU>  // WPU warps hold a head's block
__global__ void __launch_bounds__(kPackWarps * 32)
k_q8_pack(Q8PackArgs a) {
  constexpr int CH = D / 8, UPC = kPackWarps / WPU;
  __shared__ uint32_t sh[kPackWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x / a.hgroups, l = blockIdx.y;
  const int h = (blockIdx.x % a.hgroups) * UPC + warp / WPU;
  const int part = (warp % WPU) * 32 + lane;  // thread of the head's block
  const int32_t src = a.src[pair], dst = a.dst[pair];
  if (src < 0 && dst < 0) return;  // (a pair that is left out)
  if (src < 0 || src >= a.n_blocks || dst < 0 || dst >= a.n_blocks8) {
    if (threadIdx.x == 0) record_error(a.status, KVC_ERR_BOUNDS);
    return;
  }
  const bool live = h < a.H;
  const int chunks = live ? a.BS * CH : 0;
  const uint16_t *pool = (blockIdx.z ? a.vpool : a.kpool) +
                         (((int64_t)l * a.n_blocks + src) * a.BS * a.H + h) * D;
  uint4 x[kPackLoads];
#pragma unroll
  for (int i = 0; i < kPackLoads; i++) {
    const int e = i * WPU * 32 + part;
    x[i] = make_uint4(0, 0, 0, 0);
    if (e < chunks) x[i] = ld_stream(pool + (int64_t)(e / CH) * a.H * D + (e % CH) * 8);
  }
  // the largest finite magnitude, as bf16 bits (their order is the values')
  uint32_t top = 0;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < kPackLoads; i++) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t a0 = w[e] & 0x7FFFu, a1 = (w[e] >> 16) & 0x7FFFu;
      odd |= a0 >= 0x7F80u || a1 >= 0x7F80u;
      top = max(top, max(a0 < 0x7F80u ? a0 : 0u, a1 < 0x7F80u ? a1 : 0u));
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (WPU > 1) {
    if (lane == 0) sh[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPU; w++) top = max(top, sh[warp / WPU * WPU + w]);
  }
  if (odd) record_error(a.status, KVC_ERR_NAN);
  if (!live) return;
  // top = m·2^x with m in [1, 2): 448 = 1.75·2^8, so s = 2^(x − 8), or twice that past 1.75
  int ex = (int)(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u);
  ex = top == 0 ? 0 : max(ex, -126);
  const float scale = __uint_as_float((uint32_t)(ex + 127) << 23);
  const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
  const int64_t at = ((int64_t)l * a.n_blocks8 + dst) * a.H + h;
  uint8_t *out = (blockIdx.z ? a.v8 : a.k8) + at * a.BS * D;
#pragma unroll
  for (int i = 0; i < kPackLoads; i++) {
    const int e = i * WPU * 32 + part;
    if (e >= chunks) break;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t y[4];
#pragma unroll
    for (int u = 0; u < 4; u++)
      y[u] = __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(w[u]) * inv, bf16_hi(w[u]) * inv),
                                      __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2 *>(out + e * 8) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
  }
  if (part == 0) (blockIdx.z ? a.vscale : a.kscale)[at] = scale;
}

}  // namespace

cudaError_t launch_q8_pack(const uint16_t *kpool, const uint16_t *vpool, int64_t n_slots,
                           uint8_t *k8, uint8_t *v8, float *kscale, float *vscale,
                           int64_t n_blocks8, const int32_t *src, const int32_t *dst, int n,
                           int L, int H, int D, int BS, int32_t *status, cudaStream_t s) {
  Q8PackArgs a{};
  a.kpool = kpool, a.vpool = vpool, a.k8 = k8, a.v8 = v8, a.kscale = kscale, a.vscale = vscale;
  a.src = src, a.dst = dst, a.status = status;
  a.n_blocks = n_slots / BS, a.n_blocks8 = n_blocks8, a.H = H, a.BS = BS;
  const int warps = (BS * D / 8 + kPackLoads * 32 - 1) / (kPackLoads * 32);
  const int wpu = warps <= 1 ? 1 : warps <= 2 ? 2 : 4;
  a.hgroups = (H * wpu + kPackWarps - 1) / kPackWarps;
  const dim3 grid((unsigned)(n * a.hgroups), (unsigned)L, 2);
  auto *kern = D == 128 ? (wpu == 1 ? k_q8_pack<128, 1> : wpu == 2 ? k_q8_pack<128, 2> : k_q8_pack<128, 4>)
                        : (wpu == 1 ? k_q8_pack<64, 1> : k_q8_pack<64, 2>);
  kern<<<grid, kPackWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
