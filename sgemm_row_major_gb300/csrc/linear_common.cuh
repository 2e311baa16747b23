// linear_common.cuh -- device helpers of the operators on BF16 layers: activations and their derivatives, the
// tensor-core instructions and tile descriptors for BF16, and what the products' epilogues share.
#pragma once

#include <type_traits>

#include "fp8_common.cuh"
#include "fp8_gemm.cuh"
#include "linear_internal.h"

namespace sgemm_impl {
namespace lin {

using f8::Chunk;
using f8::copies_arrive;
using f8::elect_one;
using f8::extent;
using f8::get_at;
using f8::kMaxE4M3;
using f8::poll_wait;
using f8::put_at;
using f8::tmem_ld32;

// ---- activations, in FP32
//
// exp(-a) is expf(), whose infinity for a below -88 makes the quotients 0; a quotient of a finite value and an infinity is
// 0 with the fast division too (2 ulp; its result is 0 for divisors above 2^126, where the true one is below 2^-100 of a).
template <int ACT>
__device__ __forceinline__ float act_of(float a) {
  if constexpr (ACT == SGEMM_ACT_RELU) return a < 0.0f ? 0.0f : a;
  else if constexpr (ACT == SGEMM_ACT_SILU) return __fdividef(a, 1.0f + expf(-a));
  else if constexpr (ACT == SGEMM_ACT_GELU) return a * (0.5f * erfcf(a * -0.70710678f));  // Phi(a) without cancellation for a < 0
  else if constexpr (ACT == SGEMM_ACT_GELU_TANH) return __fdividef(a, 1.0f + expf(-1.59576912f * fmaf(0.044715f * a * a, a, a)));
  else return a;
}

// f(the activation as a constant): one branch around a loop over elements, whose steps then overlap.
template <typename F>
__device__ __forceinline__ void with_act(int act, const F& f) {
  switch (act) {
    case SGEMM_ACT_RELU: return f(std::integral_constant<int, SGEMM_ACT_RELU>{});
    case SGEMM_ACT_SILU: return f(std::integral_constant<int, SGEMM_ACT_SILU>{});
    case SGEMM_ACT_GELU: return f(std::integral_constant<int, SGEMM_ACT_GELU>{});
    case SGEMM_ACT_GELU_TANH: return f(std::integral_constant<int, SGEMM_ACT_GELU_TANH>{});
    default: return f(std::integral_constant<int, SGEMM_ACT_NONE>{});
  }
}

// The activation f and its derivative df.  Where a factor of a product has become 0 the product's limit is taken (a s (1 - s)
// and a phi(a) are 0 for a beyond their range, infinite a among them).
template <int ACT>
__device__ __forceinline__ void act_grad(float a, float& f, float& df) {
  if constexpr (ACT == SGEMM_ACT_RELU) {
    f = a < 0.0f ? 0.0f : a;
    df = a > 0.0f ? 1.0f : a <= 0.0f ? 0.0f : a;  // NaN stays NaN
  } else if constexpr (ACT == SGEMM_ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + expf(-a));
    const float t = s * (1.0f - s);
    f = a * s;
    df = t == 0.0f ? s : fmaf(a, t, s);
  } else if constexpr (ACT == SGEMM_ACT_GELU) {
    const float c = 0.5f * erfcf(a * -0.70710678f), phi = 0.39894228f * expf(-0.5f * a * a);
    f = a * c;
    df = phi == 0.0f ? c : fmaf(a, phi, c);
  } else if constexpr (ACT == SGEMM_ACT_GELU_TANH) {
    const float a2 = a * a;
    const float s = __fdividef(1.0f, 1.0f + expf(-1.59576912f * fmaf(0.044715f * a2, a, a)));
    const float t = s * (1.0f - s);
    f = a * s;
    df = t == 0.0f ? s : fmaf(a * t, 1.59576912f * fmaf(0.134145f, a2, 1.0f), s);
  } else {
    f = a;
    df = 1.0f;
  }
}

// ---- tensor cores
//
// A tile of an operand for 64 k is at most 16 KB of shared memory with the 128-byte swizzle, in either order:
//   K-major: output rows of 64 k, one row per 128 bytes; a step of 16 k starts 32 bytes further along the rows;
//   MN-major: blocks of 64 k-rows of 64 output rows each (128 bytes), 8 KB; a step of 16 k starts 16 rows (2048 bytes)
//   further down, the next 64 output rows lie in the next block.
// Both have 8-row atoms 1024 bytes apart.  Only the low word of a descriptor depends on the tile.
constexpr int kBlockBytes = 64 * 128;
constexpr uint32_t kDescHi = (1024u >> 4)    // stride offset: next 8 rows of the tile
                             | (1u << 14)    // descriptor version for tcgen05
                             | (2u << 29);   // 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_byte_addr) {
  return ((smem_byte_addr & 0x3FFFFu) >> 4) | ((uint32_t)(kBlockBytes >> 4) << 16);  // leading offset: next 64 output rows (MN-major)
}
__device__ __forceinline__ uint64_t make_desc(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
__device__ __forceinline__ uint32_t step_of(int mn_major) { return mn_major ? (2048u >> 4) : (32u >> 4); }

__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// K tiles summed in one accumulator before they are added to sums in FP32 registers: the tensor cores' own accumulation is not
// round-to-nearest and drifts by about 1.2e-8 of the sum per instruction of 16 k; 32 of them stay below 4e-7.
constexpr int kFold = 8;

// ---- what an epilogue reads and writes

// Two consecutive values as BF16, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ bool d_ok(const LinearOut& o, int which, int64_t row, int64_t col, int64_t n) {
  return in_range(o.guard.fault, o.guard.word, f8::kSiteOut, row * o.ldd[which] + col, n, extent(o.M, o.ldd[which], o.N));
}
__device__ __forceinline__ bool r_ok(const LinearOut& o, int64_t row, int64_t col, int64_t n) {
  return in_range(o.guard.fault, o.guard.word, f8::kSiteIn, row * o.ldr + col, n, extent(o.M, o.ldr, o.N));
}
__device__ __forceinline__ bool kept_ok(const LinearOut& o, int which, int64_t row, int64_t col, int64_t n) {
  return in_range(o.guard.fault, o.guard.word, f8::kSiteCodes, row * o.kept[which].ld + col, n, extent(o.M, o.kept[which].ld, o.N));
}
// The scale of group `group` of a row of a kept 8-bit matrix.
__device__ __forceinline__ void put_scale(const LinearOut& o, int which, int64_t row, int64_t group, float s) {
  const LinearKept& k = o.kept[which];
  if (in_range(o.guard.fault, o.guard.word, f8::kSiteScale, row * k.lds + group, 1, extent(o.M, k.lds, (o.N + 127) / 128)))
    k.scale[row * k.lds + group] = s;
}

}  // namespace lin
}  // namespace sgemm_impl
