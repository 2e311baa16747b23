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

// ---- activations, in FP32, two values at a time (packed arithmetic: the epilogues and the gradient kernel are bound by the
// number of instructions as much as by the memory)
//
// The exponential is ex2.approx.ftz (2^-22 of its result; 0 or infinity beyond its range), the reciprocal rcp.approx.ftz (1 ulp,
// 0 for an infinity), so a quotient of a finite value and an infinity is 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float2 rcp(float2 x) { return make_float2(rcp(x.x), rcp(x.y)); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
// c where k is 0, else x
__device__ __forceinline__ float2 unless0(float2 k, float2 c, float2 x) { return make_float2(k.x == 0.0f ? c.x : x.x, k.y == 0.0f ? c.y : x.y); }

// e = exp(-a^2 / 2) and Phi(a).  Phi(-|a|) = e P(t), t = 1 / (1 + 0.28284273 |a|), with P of degree 9 fitted to
// exp(a^2 / 2) Phi(-|a|) over all a (least maximum of the relative error, 1.3e-7; 4.4e-7 evaluated in FP32), so that small
// values of Phi keep their relative accuracy.
__device__ __forceinline__ float2 normal_integral(float2 a, float2& e) {
  const float2 m = make_float2(fabsf(a.x), fabsf(a.y));
  const float2 t = rcp(fma(m, both(0.28284273f), both(1.0f)));
  e = ex2(mul(mul(a, both(-0.72134752f)), a));
  float2 q = both(0.025131345f);
  q = fma(q, t, both(-0.09145177f));
  q = fma(q, t, both(0.08454426f));
  q = fma(q, t, both(-0.00280497f));
  q = fma(q, t, both(0.070716225f));
  q = fma(q, t, both(0.08427088f));
  q = fma(q, t, both(0.10392137f));
  q = fma(q, t, both(0.112834804f));
  q = fma(q, t, both(0.11283793f));
  q = mul(mul(q, t), e);
  return make_float2(a.x >= 0.0f ? 1.0f - q.x : q.x, a.y >= 0.0f ? 1.0f - q.y : q.y);
}

// 1 / (1 + exp(-a)) and, for GELU's tanh form, 1 / (1 + exp(-2 u))
__device__ __forceinline__ float2 sigmoid(float2 a) { return rcp(add(ex2(mul(a, both(-1.44269504f))), both(1.0f))); }
__device__ __forceinline__ float2 sigmoid_2u(float2 a, float2 a2) {
  return rcp(add(ex2(mul(a, fma(a2, both(-0.10294324f), both(-2.3022082f)))), both(1.0f)));
}

template <int ACT>
__device__ __forceinline__ float2 act_of(float2 a) {
  if constexpr (ACT == SGEMM_ACT_RELU) return make_float2(a.x < 0.0f ? 0.0f : a.x, a.y < 0.0f ? 0.0f : a.y);
  else if constexpr (ACT == SGEMM_ACT_SILU) return mul(a, sigmoid(a));
  else if constexpr (ACT == SGEMM_ACT_GELU) {
    float2 e;
    return mul(a, normal_integral(a, e));
  } else if constexpr (ACT == SGEMM_ACT_GELU_TANH) return mul(a, sigmoid_2u(a, mul(a, a)));
  else return a;
}

// f(the activation as a constant): one branch around a loop over elements, whose steps then overlap.
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, const F& f) {
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
__device__ __forceinline__ void act_grad(float2 a, float2& f, float2& df) {
  if constexpr (ACT == SGEMM_ACT_RELU) {
    f = act_of<ACT>(a);
    df = make_float2(a.x > 0.0f ? 1.0f : a.x <= 0.0f ? 0.0f : a.x, a.y > 0.0f ? 1.0f : a.y <= 0.0f ? 0.0f : a.y);  // NaN stays NaN
  } else if constexpr (ACT == SGEMM_ACT_SILU) {
    const float2 s = sigmoid(a), t = fma(make_float2(-s.x, -s.y), s, s);
    f = mul(a, s);
    df = unless0(t, s, fma(a, t, s));
  } else if constexpr (ACT == SGEMM_ACT_GELU) {
    float2 e;
    const float2 c = normal_integral(a, e);
    f = mul(a, c);
    df = unless0(e, c, fma(mul(a, both(0.39894228f)), e, c));
  } else if constexpr (ACT == SGEMM_ACT_GELU_TANH) {
    const float2 a2 = mul(a, a);
    const float2 s = sigmoid_2u(a, a2), t = fma(make_float2(-s.x, -s.y), s, s);
    f = mul(a, s);
    df = unless0(t, s, fma(mul(a, t), fma(a2, both(0.21406445f), both(1.5957691f)), s));
  } else {
    f = a;
    df = both(1.0f);
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

// Copies one operand's tile of `rows` output rows (at most 128) and 64 k: boxes of 64 output rows in either order, one 8 KB
// block behind the other.
template <typename Load>
__device__ __forceinline__ void load_part(const Load& load, uint32_t dst, const CUtensorMap* map, int mn_major, int mn0, int k0, int rows) {
#pragma unroll
  for (int i = 0; i < (rows > 64 ? 2 : 1); ++i)
    load(dst + (uint32_t)(i * kBlockBytes), map, mn_major ? mn0 + 64 * i : k0, mn_major ? k0 : mn0 + 64 * i);
}
// Bytes that it copies.
__host__ __device__ constexpr uint32_t part_bytes(int mn_major, int rows) { return mn_major ? (rows > 64 ? 2u : 1u) * kBlockBytes : (uint32_t)rows * 128u; }

// ---- what an epilogue reads and writes

// Two consecutive values as BF16, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four elements of a BF16 row, n of them there.
__device__ __forceinline__ void get4(const __nv_bfloat16* p, int n, bool vec, float (&x)[4]) {
  if (vec && n == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xFFFF0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e < n ? __bfloat162float(p[e]) : 0.0f;
  }
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, int n, bool vec, const float (&x)[4]) {
  if (vec && n == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = __float2bfloat16_rn(x[e]);
  }
}

__device__ __forceinline__ bool d_ok(const LinearOut& o, const LinearJob& j, int64_t row, int64_t col, int64_t n) {
  return in_range(o.guard.fault, o.guard.word, f8::kSiteOut, row * j.ldd + col, n, extent(j.M, j.ldd, j.N));
}
__device__ __forceinline__ bool r_ok(const LinearOut& o, const LinearJob& j, int64_t row, int64_t col, int64_t n) {
  return in_range(o.guard.fault, o.guard.word, f8::kSiteIn, row * o.ldr + col, n, extent(j.M, o.ldr, j.N));
}
__device__ __forceinline__ bool kept_ok(const LinearOut& o, const LinearJob& j, int which, int64_t row, int64_t col, int64_t n) {
  return in_range(o.guard.fault, o.guard.word, f8::kSiteCodes, row * o.kept[which].ld + col, n, extent(j.M, o.kept[which].ld, j.N));
}
// The scale of group `group` of a row of a kept 8-bit matrix.
__device__ __forceinline__ void put_scale(const LinearOut& o, const LinearJob& j, int which, int64_t row, int64_t group, float s) {
  const LinearKept& k = o.kept[which];
  if (in_range(o.guard.fault, o.guard.word, f8::kSiteScale, row * k.lds + group, 1, extent(j.M, k.lds, (j.N + 127) / 128)))
    k.scale[row * k.lds + group] = s;
}

// Four columns of a row of D, n of them there.
__device__ __forceinline__ void put_row(const LinearOut& o, const LinearJob& j, int row, int col, int n, const float (&v)[4]) {
  if (!d_ok(o, j, row, col, n)) return;
  if (j.f32) {
    float* d = static_cast<float*>(j.d) + (int64_t)row * j.ldd + col;
    if (j.d_vec && n == 4) {
      *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) d[e] = v[e];
    }
  } else {
    put4(static_cast<__nv_bfloat16*>(j.d) + (int64_t)row * j.ldd + col, n, j.d_vec, v);
  }
}

}  // namespace lin
}  // namespace sgemm_impl
