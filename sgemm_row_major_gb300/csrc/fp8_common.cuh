// fp8_common.cuh -- device helpers shared by the 8-bit operators: conversion to codes, the scale
// of a group, and chunk loads and stores of FP32 / BF16 rows.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "device_utils.cuh"
#include "fp8_internal.h"
#include "sgemm_fp8.h"

namespace sgemm_impl {
namespace f8 {

constexpr float kMaxE4M3 = 448.0f, kMaxE5M2 = 57344.0f;
constexpr float kMaxFloat = 3.402823466e38f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: the smallest scale, whose reciprocal is finite

// What the debug build's checks report of an index outside its buffer (they follow enum BoundsSite).
enum Fp8Site : unsigned {
  kSiteIn = 16,      // X, R, W, dY, H, dH, C read
  kSiteOut = 17,     // H, Y, dX, D, dW written
  kSiteCodes = 18,   // codes written or copied
  kSiteScale = 19,   // scales
  kSiteRowStat = 20, // rstd
  kSiteLogits = 21,  // logits
  kSitePart = 22     // the workspace: partial sums, inner values, routing
};

// One element at index i of the n at p (the check is the constant true in the normal build).
template <typename T>
__device__ __forceinline__ T get_at(const Guard& g, unsigned site, const T* p, int64_t i, int64_t n) {
  return in_range(g.fault, g.word, site, i, 1, n) ? p[i] : T();
}
template <typename T>
__device__ __forceinline__ void put_at(const Guard& g, unsigned site, T* p, int64_t i, int64_t n, T v) {
  if (in_range(g.fault, g.word, site, i, 1, n)) p[i] = v;
}
// Elements from the first to one past the last of a matrix.
__device__ __forceinline__ int64_t extent(int64_t rows, int64_t ld, int64_t cols) { return (rows - 1) * ld + cols; }

// |x| where it is finite, else 0: what counts towards a group's largest value.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= kMaxFloat ? a : 0.0f;
}

// A group's scale.  top * kMinScale is far below any value that matters, so a group of zeros
// (and one without finite values) simply gets the smallest scale.
__device__ __forceinline__ float group_scale(float amax, float top) { return fmaxf(__fdiv_rn(amax, top), kMinScale); }

// Two values (already divided by their scale, so at most `top` a rounding or two beyond it when
// finite) to two codes, the first in the low byte; round to nearest even, NaN for a non-finite
// value (the conversion alone would turn an infinity into the largest finite code).
// CHECK = false: no value is infinite (a NaN needs no test).
template <bool CHECK>
__device__ __forceinline__ uint32_t codes2(float a, float b, bool e5m2) {
  if (CHECK) {
    const float nan = __int_as_float(0x7FFFFFFF);
    a = fabsf(a) <= kMaxFloat ? a : nan;
    b = fabsf(b) <= kMaxFloat ? b : nan;
  }
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, e5m2 ? __NV_E5M2 : __NV_E4M3);
}

template <bool CHECK>
__device__ __forceinline__ uint32_t codes4(const float* v, const float* inv, bool e5m2) {
  return codes2<CHECK>(v[0] * inv[0], v[1] * inv[1], e5m2) | (codes2<CHECK>(v[2] * inv[2], v[3] * inv[3], e5m2) << 16);
}

// V consecutive elements as stored (16 bytes): 4 floats or 8 BF16 values.
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
  static constexpr int V = 4;
  uint4 raw;
  __device__ __forceinline__ void get(float* v) const {
    v[0] = __uint_as_float(raw.x);
    v[1] = __uint_as_float(raw.y);
    v[2] = __uint_as_float(raw.z);
    v[3] = __uint_as_float(raw.w);
  }
  __device__ __forceinline__ void put(const float* v) {
    raw = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int V = 8;
  uint4 raw;
  __device__ __forceinline__ void get(float* v) const {  // BF16 is the upper half of an FP32 value
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void put(const float* v) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    raw = make_uint4(u[0], u[1], u[2], u[3]);
  }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A matrix that chunks are loaded from or stored to: `end` is past its last element.
template <typename T>
struct Rows {
  const T *base, *end;
  const Guard& guard;
  __device__ __forceinline__ Rows(const void* p, int64_t rows, int64_t ld, int64_t cols, const Guard& g)
      : base(static_cast<const T*>(p)), end(static_cast<const T*>(p) + extent(rows, ld, cols)), guard(g) {}
  __device__ __forceinline__ bool holds(unsigned site, const T* p, int64_t n) const {
    return n <= 0 || in_range(guard.fault, guard.word, site, p - base, n, end - base);
  }
};

// A chunk of elements [0, n) at p, zeros beyond n, in two steps: load() sends for it, get() waits for it
// (so that several are on their way at once).  VEC: p is 16-byte aligned and n is 0 or >= V.  Otherwise
// any p that is aligned to its type (rows of an odd number of columns begin anywhere): FP32 element by
// element; BF16 as the 16-byte units that p lies in, where they are inside the matrix, shifted into place
// (element by element the norm of 8192 x 4095 took 113 us, so 66 us).
template <typename T, bool VEC>
struct Loading {
  static constexpr int V = Chunk<T>::V;
  uint4 a, b;
  uint32_t off;  // bytes to shift by
  int left;
  __device__ __forceinline__ void load(const T* p, int64_t n, const Rows<T>& m) {
    a = b = make_uint4(0u, 0u, 0u, 0u);
    if (!m.holds(kSiteIn, p, VEC && n > 0 ? (int64_t)V : min((int64_t)V, n))) n = 0;
    if (VEC) {
      if (n > 0) a = *reinterpret_cast<const uint4*>(p);
      return;
    }
    left = (int)max((int64_t)0, min((int64_t)V, n));
    if (sizeof(T) == 4) {
      const uint32_t* e = reinterpret_cast<const uint32_t*>(p);
      a.x = left > 0 ? e[0] : 0u;
      a.y = left > 1 ? e[1] : 0u;
      a.z = left > 2 ? e[2] : 0u;
      a.w = left > 3 ? e[3] : 0u;
      return;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), unit = at & ~(uintptr_t)15;
    off = (uint32_t)(at - unit);
    if (left == 0) return;
    const bool two = off + left * sizeof(T) > 16u;
    if (unit >= reinterpret_cast<uintptr_t>(m.base) && unit + (two ? 32 : 16) <= reinterpret_cast<uintptr_t>(m.end)) {
      a = *reinterpret_cast<const uint4*>(unit);
      if (two) b = *reinterpret_cast<const uint4*>(unit + 16);
    } else {
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < left ? to_float(p[i]) : 0.0f;
      Chunk<T> c;
      c.put(v);  // exact: every value came from T
      a = c.raw;
      off = 0u;
    }
  }
  __device__ __forceinline__ Chunk<T> get() const {
    Chunk<T> c;
    if (VEC || sizeof(T) == 4) {
      c.raw = a;
      return c;
    }
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = off & 8u ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = off & 4u ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8u * (off & 2u));
    if (left < V) {
      constexpr int kPer = 4 / sizeof(T);  // elements per word
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int here = left - i * kPer;
        w[i] = here <= 0 ? 0u : here < kPer ? w[i] & 0xFFFFu : w[i];
      }
    }
    c.raw = make_uint4(w[0], w[1], w[2], w[3]);
    return c;
  }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* p, const float* v, int64_t n, const Rows<T>& m) {
  constexpr int V = Chunk<T>::V;
  if (!m.holds(kSiteOut, p, VEC && n > 0 ? (int64_t)V : min((int64_t)V, n))) return;
  if (VEC ? n > 0 : n >= V && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    Chunk<T> c;
    c.put(v);
    *reinterpret_cast<uint4*>(p) = c.raw;
  } else if (!VEC) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) from_float(p + i, v[i]);
  }
}

// V codes (4 or 8) of one chunk, value i times inv[i].
template <int V, bool CHECK>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* v, const float* inv, int64_t n, bool e5m2,
                                            const Rows<uint8_t>& m) {
  if (!m.holds(kSiteCodes, p, min((int64_t)V, n))) return;
  uint32_t u[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) u[i] = codes4<CHECK>(v + 4 * i, inv + 4 * i, e5m2);
  if (n >= V && (reinterpret_cast<uintptr_t>(p) & (V - 1)) == 0) {
    if (V == 4) *reinterpret_cast<uint32_t*>(p) = u[0];
    else        *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[V / 4 - 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = (uint8_t)(u[i / 4] >> (8 * (i % 4)));
  }
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

}  // namespace f8
}  // namespace sgemm_impl
