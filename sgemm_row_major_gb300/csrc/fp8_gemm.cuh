// fp8_gemm.cuh -- device helpers of the block-scaled 8-bit products (kernel_fp8_pair.cuh,
// kernel_fp8_short.cu): tile descriptors, the tensor-core instructions, and the output's rows.
#pragma once

#include <type_traits>

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
// Only the low word of a descriptor depends on the tile.
constexpr uint32_t kDescHi = (1024u >> 4)    // stride offset: next 8 rows of the tile
                             | (1u << 14)    // descriptor version for tcgen05
                             | (2u << 29);   // 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_byte_addr) {
  return ((smem_byte_addr & 0x3FFFFu) >> 4) |
         ((1024u >> 4) << 16);  // leading offset: next 128 output rows of an MN-major tile (never reached)
}
__device__ __forceinline__ uint64_t make_desc(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
__device__ __forceinline__ uint32_t step_of(int mn_major) { return mn_major ? (4096u >> 4) : (32u >> 4); }

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

// Whether a barrier phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Bounded wait of a whole warp for a barrier phase, for waits that are short: every lane polls (each
// has its own acquire), the clock is read only now and then, and nothing is called, so the sums that
// the fold keeps in registers stay there.  Warp-uniform.
__device__ __forceinline__ bool poll_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
  bool ok = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
#pragma unroll 1
      for (int i = 0; i < 32 && !ok; ++i) ok = mbar_try_wait(bar, parity);
      if (ok || global_timer_ns() - t0 > timeout_ns) break;
    }
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}

// True in one lane of a converged warp, the same one every time.  The warps that issue copies and
// products run their loops with all lanes and issue under this predicate: operands that the compiler
// can see to be the same in every lane stay in uniform registers, while in a branch of one lane each
// operand of each instruction is moved there first (a group of four products then took 700 cycles
// to issue).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// N (16 or 32) consecutive columns.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  static_assert(N == 16 || N == 32, "columns at a time");
  if constexpr (N == 32) tmem_ld32(taddr, v);
  else                   tmem_ld16(taddr, v);
}

// 16 rows x 32 columns of this warp's TMEM lanes from taddr's lane on, as the tensor cores' own fragments
// lie: thread t receives of rows t / 4 and t / 4 + 8, for each 8 columns, columns 2 (t % 4) and the next
// (v[4 j], v[4 j + 1] of the first row, v[4 j + 2], v[4 j + 3] of the second).
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Element i of the n at src from global to shared memory, asynchronously.
__device__ __forceinline__ void copy4_async(const Guard& g, unsigned site, uint32_t dst, const float* src, int64_t i, int64_t n) {
  if (!in_range(g.fault, g.word, site, i, 1, n)) return;
  src += i;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` (one of the arrivals it counts) when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int REGS>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}

// Scales that an operand of mn rows (columns) of op(X) has, from the first to one past the last.
__device__ __forceinline__ int64_t extent(const Fp8Scales& s, int mn, int groups) {
  return ((mn - 1) >> s.shift) * s.si + (groups - 1) * s.sk + 1;
}

// Whether `n` elements of C (D) from row `row`, column `col` on lie in it.
__device__ __forceinline__ bool c_holds(const Fp8Out& o, int64_t row, int64_t col, int64_t n) {
  return in_range(o.guard.fault, o.guard.word, kSiteIn, row * o.ldc + col, n, extent(o.M, o.ldc, o.N));
}
__device__ __forceinline__ bool d_holds(const Fp8Out& o, int64_t row, int64_t col, int64_t n) {
  return in_range(o.guard.fault, o.guard.word, kSiteOut, row * o.ldd + col, n, extent(o.M, o.ldd, o.N));
}

__device__ __forceinline__ float read_c(const Fp8Out& o, int64_t row, int64_t col) {
  if (!c_holds(o, row, col, 1)) return 0.0f;
  const int64_t i = row * o.ldc + col;
  return o.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(o.C)[i]) : static_cast<const float*>(o.C)[i];
}

// One element of D from its sum.
__device__ __forceinline__ void store_one(const Fp8Out& o, int64_t row, int64_t col, float v) {
  float x = o.alpha * v;
  if (o.beta != 0.0f) x = fmaf(o.alpha, v, o.beta * read_c(o, row, col));
  if (!d_holds(o, row, col, 1)) return;
  const int64_t i = row * o.ldd + col;
  if (o.bf16) static_cast<__nv_bfloat16*>(o.D)[i] = __float2bfloat16_rn(x);
  else        static_cast<float*>(o.D)[i] = x;
}

// How the output is written, known where the kernel is chosen (the caller holds 128 sums in registers
// meanwhile; all cases in one kernel cost 9% at 8192^3).
enum Output {
  kOutPlain = 0,  // beta == 0, aligned rows of whole 16 bytes: TMA
  kOutAdd = 1,    // beta != 0, aligned rows
  kOutAny = 2     // any alignment and beta
};

// Rows of one lane of an aligned piece, 4 rows apart, all of them in D: no tests between the
// accesses, so that the loads of a batch are in flight together.
template <bool BF16>
__device__ __forceinline__ void store_aligned_rows(const Fp8Out& o, int64_t row, int64_t col, const float* v,
                                                   int pitch) {
  constexpr int kBatch = 8;  // all of them: each batch waits for C once
  using T = typename std::conditional<BF16, uint2, float4>::type;  // 4 elements
  constexpr int kSize = BF16 ? 2 : 4;
  char* d = static_cast<char*>(o.D) + (row * o.ldd + col) * kSize;
  const char* c = static_cast<const char*>(o.C) + (row * o.ldc + col) * kSize;
  const int64_t dstep = 4 * o.ldd * kSize, cstep = 4 * o.ldc * kSize;
  if (!c_holds(o, row, col, 28 * o.ldc + 4) || !d_holds(o, row, col, 28 * o.ldd + 4)) return;
#pragma unroll
  for (int r0 = 0; r0 < 8; r0 += kBatch) {
    float4 x[kBatch];
    T old[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      x[k] = *reinterpret_cast<const float4*>(v + 4 * (r0 + k) * pitch);
      old[k] = *reinterpret_cast<const T*>(c);
      c += cstep;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      float4 u;
      if constexpr (BF16)
        u = make_float4(__uint_as_float(old[k].x << 16), __uint_as_float(old[k].x & 0xFFFF0000u),
                        __uint_as_float(old[k].y << 16), __uint_as_float(old[k].y & 0xFFFF0000u));
      else
        u = old[k];
      const float4 y = make_float4(fmaf(o.alpha, x[k].x, o.beta * u.x), fmaf(o.alpha, x[k].y, o.beta * u.y),
                                   fmaf(o.alpha, x[k].z, o.beta * u.z), fmaf(o.alpha, x[k].w, o.beta * u.w));
      if constexpr (BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), b = __floats2bfloat162_rn(y.z, y.w);
        *reinterpret_cast<T*>(d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      } else {
        *reinterpret_cast<T*>(d) = y;
      }
      d += dstep;
    }
  }
}

// One column of a piece, element by element: `rows` rows from row0, what C holds kBatch rows at a time.
template <typename T, int kBatch>
__device__ __forceinline__ void store_rows_any(const Fp8Out& o, int row0, int col, int rows, bool add, const float* v,
                                               int pitch) {
  T* d = static_cast<T*>(o.D) + (int64_t)row0 * o.ldd + col;
  const T* c = static_cast<const T*>(o.C) + (add ? (int64_t)row0 * o.ldc + col : 0);
  if (rows > 0 && ((add && !c_holds(o, row0, col, (rows - 1) * o.ldc + 1)) || !d_holds(o, row0, col, (rows - 1) * o.ldd + 1))) return;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += kBatch) {
    T old[kBatch];
    if (add) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k, c += o.ldc)
        if (r0 + k < rows) old[k] = *c;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k, v += pitch, d += o.ldd)
      if (r0 + k < rows) from_float(d, add ? fmaf(o.alpha, *v, o.beta * to_float(old[k])) : o.alpha * *v);
  }
}

// A 32-row x 32-column piece of D from its sums in shared memory (`piece`, `pitch` words from row to
// row), by one warp.  With aligned rows eight lanes hold 32 consecutive columns (128 bytes of FP32, 64
// of BF16) of 4 rows at a time, otherwise (and at D's edges) a row is written by lanes with one element
// each; what C holds is loaded for several rows before any is used.
template <int OUT>
__device__ __forceinline__ void store_piece(const Fp8Out& o, int row0, int col0, const float* piece, int pitch) {
  const int lane = threadIdx.x & 31;
  if (OUT == kOutAdd && col0 + 32 <= o.N && row0 + 32 <= o.M) {
    const int at = 4 * (lane & 7), row = lane >> 3;
    const float* v = piece + row * pitch + at;
    if (o.bf16) store_aligned_rows<true>(o, row0 + row, col0 + at, v, pitch);
    else        store_aligned_rows<false>(o, row0 + row, col0 + at, v, pitch);
    return;
  }
  const int col = col0 + lane;
  if (col >= o.N) return;
  const bool add = OUT == kOutAdd || o.beta != 0.0f;
  const int rows = min(32, o.M - row0);
  constexpr int kBatch = OUT == kOutAny ? 32 : 8;  // (at the edges only, where registers are short)
  if (o.bf16) store_rows_any<__nv_bfloat16, kBatch>(o, row0, col, rows, add, piece + lane, pitch);
  else        store_rows_any<float, kBatch>(o, row0, col, rows, add, piece + lane, pitch);
}

}  // namespace f8
}  // namespace sgemm_impl
