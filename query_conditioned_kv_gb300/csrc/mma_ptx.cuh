// mma_ptx.cuh — building blocks of the kernels that stream paged rows into
// tensor-core products (tree_attn.cu, attn_mass.cu): cp.async and mma.sync,
// tcgen05 and TMA issued under a predicate, tensor maps of the pools and of
// the queries, the shared-memory row layout, and block-wide sums and searches
// over the requests of a batch.
#pragma once

#include "tc_ptx.cuh"

namespace kvc {
namespace {


__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}


// Byte offset of 16-byte chunk c of row `row` (rows of D elements): chunks
// are permuted by the row so that ldmatrix's eight rows hit distinct banks.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int c) {
  return (uint32_t)(row * D * 2 + ((c ^ (row & 7)) << 4));
}

// tcgen05.mma / commit by the lanes with `lead` set (one of the warp); the
// whole warp must execute it.
__device__ __forceinline__ void mma_bf16_if(uint32_t lead, uint32_t d_tmem, uint64_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit_if(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          bar),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_if(uint32_t lead, uint32_t dst, const CUtensorMap *map,
                                               int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %6, 0;\n"
      " @q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(lead)
      : "memory");
}
// The same value in every lane, for the compiler too.
__device__ __forceinline__ uint32_t uniform32(uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }
__device__ __forceinline__ uint64_t uniform64(uint64_t x) {
  return (uint64_t)uniform32((uint32_t)(x >> 32)) << 32 | uniform32((uint32_t)x);
}

// 16 TMEM lanes × 64 columns (16x256b): register 4k + j of thread t holds lane
// t/4 + 8·(j ≥ 2), column 8k + 2·(t%4) + (j & 1).
__device__ __forceinline__ void tmem_frag8(uint32_t taddr, uint32_t (&r)[32]) {
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

// The same with 32 columns.
__device__ __forceinline__ void tmem_frag4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Boxes of `box` consecutive slots of one head, 64 columns, 128-byte swizzle.
inline bool pool_map(CUtensorMap *m, const void *pool, int64_t n_slots, int H, int D, int box) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)n_slots};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
  cuuint32_t bx[3] = {64, 1, (cuuint32_t)box}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(pool), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes of `nodes` consecutive rows of q, the G heads of one group, 64 columns.
inline bool q_map(CUtensorMap *m, const void *q, int64_t n_q, int Hq, int D, int G, int nodes) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)n_q};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2};
  cuuint32_t bx[3] = {64, (cuuint32_t)G, (cuuint32_t)nodes}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// p / BS for 0 ≤ p < 2^24 and BS ≤ 64, from page_inverse(BS) = ⌈2^32 / BS⌉: the
// product's error, p·(⌈2^32/BS⌉·BS − 2^32) < 2^30, stays below 2^32.
__device__ __forceinline__ int page_of(int p, uint32_t inverse) {
  return inverse ? (int)__umulhi((uint32_t)p, inverse) : p;
}
inline uint32_t page_inverse(int BS) {
  return BS == 1 ? 0u : (uint32_t)(((1ull << 32) + BS - 1) / BS);
}

// Another CTA's shared memory (addr from mapa).
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(addr)
               : "memory");
  return v;
}

// Maximum over the CTA (a multiple of 32 threads); every thread gets it.  sh: 32
// words of scratch, free again on return.
__device__ __forceinline__ int64_t block_max(int64_t v, int64_t *sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max(v, (int64_t)__shfl_xor_sync(0xFFFFFFFFu, v, o));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
  for (int w = 1; w < (int)(blockDim.x >> 5); w++) v = max(v, sh[w]);
  __syncthreads();
  return v;
}

// x / y for x ≥ 0, y > 0 (64-bit division is a long call: most sizes fit 32 bits).
__device__ __forceinline__ int64_t div64(int64_t x, int64_t y) {
  return x >> 32 || y >> 32 ? x / y : (uint32_t)x / (uint32_t)y;
}

// Σ size(i) over [0, n), and which element holds place t of the sum.  By every
// warp for itself: a short kernel's beginning is latency, and barriers between
// its steps would add to it.
struct WarpSums {
  int64_t total;
  int64_t mine, upto;  // the lane's among the first 32: its size, the sum up to and with it
};
__device__ __forceinline__ int64_t warp_prefix(int64_t x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}
template <class F>
__device__ __forceinline__ WarpSums warp_sums(int n, F size) {
  const int lane = threadIdx.x & 31;
  WarpSums w;
  w.mine = lane < n ? size(lane) : 0;
  w.upto = warp_prefix(w.mine);
  w.total = __shfl_sync(0xFFFFFFFFu, w.upto, 31);
  if (n > 32) {
    int64_t x = 0;
#pragma unroll 4
    for (int i = 32 + lane; i < n; i += 32) x += size(i);
    w.total += __shfl_sync(0xFFFFFFFFu, warp_prefix(x), 31);
  }
  return w;
}
// The element i whose interval [Σ_{<i}, Σ_{≤i}) holds t < total, and Σ_{<i}.
template <class F>
__device__ __forceinline__ void warp_find(const WarpSums &w, int n, int64_t t, F size, int &found,
                                          int64_t &before) {
  int64_t mine = w.mine, upto = w.upto, carry = 0;
  for (int i0 = 0;;) {
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, t < carry + upto);
    if (past || i0 + 32 >= n) {
      const int at = past ? __ffs(past) - 1 : 0;
      found = i0 + at;
      before = carry + __shfl_sync(0xFFFFFFFFu, upto - mine, at);
      return;
    }
    carry += __shfl_sync(0xFFFFFFFFu, upto, 31);
    i0 += 32;
    const int i = i0 + (int)(threadIdx.x & 31);
    mine = i < n ? size(i) : 0;
    upto = warp_prefix(mine);
  }
}

}  // namespace
}  // namespace kvc
