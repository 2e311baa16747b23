// fp8_gemm.cuh -- device helpers of the block-scaled 8-bit products (kernel_fp8_pair.cu,
// kernel_fp8_short.cu): tile descriptors, the tensor-core instructions, and the output's rows.
#pragma once

#include "fp8_common.cuh"
#include "fp8_internal.h"
#include "kernel_tc_common.cuh"

namespace sgemm_impl {
namespace f8 {

// A tile of an operand for one group of 128 k is 16 KB or less of shared memory, loaded by one TMA
// box with the 128-byte swizzle, in either order:
//   K-major: rows (of the output) of 128 k, one row per 128 bytes;
//   MN-major: k-rows of 128 output rows each, one k per 128 bytes.
// Both have 8-row atoms 1024 bytes apart; a tensor-core step of 32 k starts 32 bytes further along a
// K-major row, 32 rows (4096 bytes) further down an MN-major tile.
__device__ __forceinline__ uint64_t tile_desc(uint32_t smem_byte_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_byte_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(1024u >> 4) << 16;  // leading offset: next 128 output rows of an MN-major tile (never reached)
  d |= (uint64_t)(1024u >> 4) << 32;  // stride offset: next 8 rows of the tile
  d |= (uint64_t)1 << 46;             // descriptor version for tcgen05
  d |= (uint64_t)2 << 61;             // 128-byte swizzle
  return d;
}
__device__ __forceinline__ uint64_t step_of(int mn_major) { return mn_major ? (4096u >> 4) : (32u >> 4); }

__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on this CTA's barrier `bar` once every tcgen05.mma this thread issued so far has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float read_c(const Fp8Out& o, int64_t i) {
  return o.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(o.C)[i]) : static_cast<const float*>(o.C)[i];
}

// One element of D from its sum.
__device__ __forceinline__ void store_one(const Fp8Out& o, int64_t row, int64_t col, float v) {
  float x = o.alpha * v;
  if (o.beta != 0.0f) x = fmaf(o.alpha, v, o.beta * read_c(o, row * o.ldc + col));
  const int64_t i = row * o.ldd + col;
  if (o.bf16) static_cast<__nv_bfloat16*>(o.D)[i] = __float2bfloat16_rn(x);
  else        static_cast<float*>(o.D)[i] = x;
}

// Columns col .. col + 7 of a row (col a multiple of 8, all below N, out.vec): 16-byte vectors.
__device__ __forceinline__ void store_eight(const Fp8Out& o, int64_t row, int64_t col, const float* v) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = o.alpha * v[e];
  if (o.bf16) {
    if (o.beta != 0.0f) {
      Chunk<__nv_bfloat16> c;
      float old[8];
      c.raw = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(o.C) + row * o.ldc + col);
      c.get(old);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(o.alpha, v[e], o.beta * old[e]);
    }
    Chunk<__nv_bfloat16> c;
    c.put(x);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o.D) + row * o.ldd + col) = c.raw;
  } else {
    if (o.beta != 0.0f) {
      const float4* c = reinterpret_cast<const float4*>(static_cast<const float*>(o.C) + row * o.ldc + col);
      const float4 a = c[0], b = c[1];
      const float old[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(o.alpha, v[e], o.beta * old[e]);
    }
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(o.D) + row * o.ldd + col);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

}  // namespace f8
}  // namespace sgemm_impl
