// kernel_fp8_pair.cuh -- block-scaled 8-bit product on CTA pairs for sm_103a (instantiated for the
// forms of the output in kernel_fp8_pair_{plain,add,any}.cu).
//
//     D = alpha * sum_g sA(i, g) sB(g, j) P_g(i, j) + beta * C,   P_g = sum over 128 k of code products
//
// Clusters of two CTAs on one TPC compute 256 x tile_n tiles (tile_n 64, 128 or 256) with
// tcgen05.mma.cta_group::2.kind::f8f6f4, M = 256, N = tile_n, K = 32, both operands from shared
// memory: each CTA holds 128 rows of A and half of the tile's columns of B.  Four such steps make
// one P_g in a fresh TMEM accumulator (two of 256 columns alternate); 8 warps per CTA read it back
// and add sA sB P_g to sums in FP32 registers, so every scale is an FP32 number and no sum is held
// in fewer bits.
//
// What bounds it: at tile_n = 256 the tensor cores need 512 cycles for a group, the folders 256 cycles of
// the FMA pipes (512 with a scale per column) and as many of the TMEM's reading width, and both run at the
// same time.  A group takes 740 cycles all the same (1080 with a scale per column): with two accumulators
// in the TMEM the chain of handing one over (the commit's arrival, the folders' first load, the last load,
// the arrival at the issuer) is longer than the other's products.  Without the fold it would be 540.
// Measured: 8192^3 with BF16 output 390 us, 2.8 PFLOP/s, in a short run and 444 us in a long one (the power
// limit); 4096^3 62 us; the gradient 4096 x 4096 x 8192 of both operands with column groups, added to FP32,
// 173 us.  Narrower tiles need 325 ns (128) and 295 ns
// (64) for a group of a half and a quarter of the products, and pay where the last round of 256-wide tiles
// would be far from full.
//
// Either operand may be stored along K or across it: the tensor core reads both orders, so a
// gradient's product takes the weights and activations as the forward pass left them.
//
// Warp 0 loads (TMA, 5 stages of 32 KB), warp 1 of the even CTA issues the products, warps 2 and 3 load
// scales a chunk of 8 groups ahead (and have what C holds brought to L2), warps 4-11 fold and write D.
// Persistent clusters take tiles round robin in an order that keeps 8 rows of tiles together (their A and
// B panels stay in L2).
#pragma once

#include <type_traits>

#include "fp8_gemm.cuh"

namespace sgemm_impl {
namespace f8 {
namespace {

using namespace tc;

constexpr int BM = 256, BMC = 128, BK = 128;
constexpr int kPart = 128 * BK;           // 16 KB: one operand's tile in one CTA
constexpr int kStageBytes = 2 * kPart;
constexpr int kStages = kFp8PairStages;
constexpr int kChunk = 8;                 // groups whose scales are loaded together
constexpr int kOutPitch = 36;             // words between the rows of a warp's 32 x 32 piece of D (16-byte accesses
                                          // by row and by column both hit 32 banks)
constexpr int kOutPitchFragments = 40;    // the same where a lane holds pairs of columns of 4 rows (8-byte accesses)
constexpr int kOutBytes = 5 * 1024;       // of shared memory per folding warp (pieces for TMA: 4 KB, 1024-byte aligned)
static_assert(32 * kOutPitch * 4 <= kOutBytes && 32 * kOutPitchFragments * 4 <= kOutBytes, "a piece of D");
constexpr int kFirstFold = 4;             // warps 0-3: loads, products, scales of A, scales of B
constexpr int kFoldWarps = 8;
constexpr int kThreads = 32 * (kFirstFold + kFoldWarps);
static_assert(kThreads == kFp8PairThreads, "the plan's figure");
// 384 threads are launched with 168 registers each; the four warps that move data give most of
// theirs to the folders: 128 x 40 + 256 x 232 = 384 x 168.  (16 folding warps with half the columns
// and 112 registers each spilled in some forms and were up to a third slower there.)
constexpr int kMoverRegs = 40, kFoldRegs = 232;
static_assert(128 * kMoverRegs + 32 * kFoldWarps * kFoldRegs <= kThreads * 168, "registers at launch");
constexpr int kMaxBufs = 4;
constexpr uint32_t kTmemCols = 512;
constexpr int kLoadCols = 32;             // accumulator columns a folder thread loads at a time

// Scales of a chunk of groups: of the CTA's 128 rows, and of the tile's columns (COLS) or its two or
// three column blocks.
template <bool COLS>
struct ScaleCfg {
  static constexpr int kB = COLS ? 256 : 4;
  static constexpr int kChunks = COLS ? 2 : 4;  // in shared memory
  static constexpr int kFloats = kChunk * (BMC + kB);
  static constexpr int kSmem = kStages * kStageBytes + kFoldWarps * kOutBytes + kChunks * kFloats * 4 + 1024;
  static_assert(kSmem + 1024 <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster,
                                              int32_t inner, int32_t outer) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(inner), "r"(outer), "r"(0)
      : "memory");
}

// One warp's 32 rows x 2N columns of D, from a row's sums in each lane, to global memory by TMA: 32
// columns at a time in D's type, rows of 64 (BF16) or 128 bytes with the swizzle of that width, so that
// the lanes' 16-byte stores to shared memory hit different banks.  Two BF16 pieces or one of FP32 fit
// in the warp's buffer; a piece is written when the copy that read its place before is done reading.  (Columns
// past D's, which TMA leaves out, begin at a multiple of 16 bytes: it writes whole units.)
// FRAGMENTS: a lane holds pairs of columns of 4 rows instead (tmem_ld_fragments).
template <bool BF16, bool FRAGMENTS, int N>
__device__ __forceinline__ void tma_out(const CUtensorMap& map, uint8_t* buf, const Fp8Out& o, int row0, int col0,
                                        const float2 (&sum)[N]) {
  const int lane = threadIdx.x & 31;
  const float2 alpha = make_float2(o.alpha, o.alpha);
  constexpr bool kTwo = BF16 && (N / 16) % 2 == 0;  // the two places alternate from tile to tile too
#pragma unroll
  for (int piece = 0; piece < N / 16; ++piece) {
    uint8_t* at = buf + (kTwo && piece % 2 ? 2048 : 0);
    if (lane == 0) {
      if (kTwo) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      else      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    __syncwarp();
    if constexpr (FRAGMENTS) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {  // 2 columns
        const int row = (lane >> 2) + 8 * (e % 4), col = 8 * (e / 4) + 2 * (lane & 3);
        const float2 x = __fmul2_rn(sum[16 * piece + e], alpha);
        if constexpr (BF16) {
          *reinterpret_cast<__nv_bfloat162*>(at + row * 64 + 16 * ((col >> 3) ^ ((row >> 1) & 3)) + 2 * (col & 7)) =
              __floats2bfloat162_rn(x.x, x.y);
        } else {
          *reinterpret_cast<float2*>(at + row * 128 + 16 * ((col >> 2) ^ (row & 7)) + 4 * (col & 3)) = x;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < (BF16 ? 4 : 8); ++e) {  // 16 bytes
        uint4 u;
        if constexpr (BF16) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = __fmul2_rn(sum[16 * piece + 4 * e + k], alpha);
            const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
            w[k] = *reinterpret_cast<const uint32_t*>(&b);
          }
          u = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          const float2 x = __fmul2_rn(sum[16 * piece + 2 * e], alpha), y = __fmul2_rn(sum[16 * piece + 2 * e + 1], alpha);
          u = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
        }
        const int chunk = BF16 ? e ^ ((lane >> 1) & 3) : e ^ (lane & 7);
        *reinterpret_cast<uint4*>(at + lane * (BF16 ? 64 : 128) + 16 * chunk) = u;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (row0 < o.M && col0 + 32 * piece < o.N)
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(&map)),
                     "r"(smem_addr(at)), "r"(col0 + 32 * piece), "r"(row0), "r"(0)
                     : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
}

// One warp: asks for what C holds of rows row0 .. row1 - 1 and `cols` columns to be brought to L2 while
// the tile's products run (the memory is hardly used then; when D is written, by all SMs at once, it is
// what they wait for).
__device__ __forceinline__ void prefetch_c(const Fp8Out& o, int row0, int row1, int col0, int cols) {
  if (o.beta == 0.0f) return;
  const int size = o.bf16 ? 2 : 4;
  const int64_t bytes = (int64_t)min(cols, o.N - col0) * size;
  for (int r = row0 + (threadIdx.x & 31); r < min(row1, o.M); r += 32) {
    const uintptr_t first = reinterpret_cast<uintptr_t>(o.C) + (uintptr_t)(((int64_t)r * o.ldc + col0) * size);
    const uintptr_t from = (first + 15) & ~(uintptr_t)15, to = (first + (uintptr_t)bytes) & ~(uintptr_t)15;
    if (from < to && c_holds(o, r, col0, bytes / size))
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(to - from)) : "memory");
  }
}

// TN: the tile's columns.  COLS: B has one scale per column (weight gradients), else one per 128
// columns.  Both are template arguments because the fold runs once per group in every folding warp: with the
// tile's width at run time its branches made it 2.5 times as long.
template <int TN, bool COLS, int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                    const __grid_constant__ CUtensorMap mapD, const __grid_constant__ Fp8PairParams p) {
  using Sc = ScaleCfg<COLS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], done[kStages];
  __shared__ __align__(8) uint64_t acc_empty[kMaxBufs];
  __shared__ __align__(8) uint64_t scale_full[Sc::kChunks], scale_empty[Sc::kChunks];
  __shared__ __align__(8) uint64_t fin;
  __shared__ uint32_t tmem_slot;

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cl = (int)cluster_id_x();
  const int groups = (p.K + BK - 1) / BK;
  const int tiles = p.tiles_m * p.tiles_n;
  const int my_tiles = cl < tiles ? (tiles - cl + p.clusters - 1) / p.clusters : 0;
  const int units = my_tiles * groups;
  constexpr int halfn = TN / 2;  // columns of B this CTA loads
  constexpr int bufs = (int)kTmemCols / TN < kMaxBufs ? (int)kTmemCols / TN : kMaxBufs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&done[s]), 1);
    }
    for (int b = 0; b < kMaxBufs; ++b) {
      mbar_init(smem_addr(&acc_empty[b]), 2 * kFoldWarps);
    }
    for (int c = 0; c < Sc::kChunks; ++c) {
      mbar_init(smem_addr(&scale_full[c]), 64);  // the threads of the two warps that load them
      mbar_init(smem_addr(&scale_empty[c]), kFoldWarps);
    }
    mbar_init(smem_addr(&fin), 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_addr(&tmem_slot), kTmemCols);
  tmem_fence_before_sync();
  cluster_sync();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  if (warp < kFirstFold) {
    fewer_registers<kMoverRegs>();
    if (warp == 0) {
      // ------------------------------------------------ loads (each CTA: its rows of A, its columns of B)
      if (lane == 0) {
        prefetch_tensormap(&mapA);
        prefetch_tensormap(&mapB);
      }
      __syncwarp();
      const uint32_t bytes = 2u * (uint32_t)(kPart + (p.b_mn ? kPart : halfn * BK));  // both CTAs'
      const uint32_t full0 = map_to_rank(smem_addr(&full[0]), 0);
      int t = 0, s = 0;
      uint32_t lap = 0;
      bool ok = true;
      for (int i = 0; ok && i < my_tiles; ++i) {
        int tm, tn;
        tile_coords(cl + i * p.clusters, p.tiles_m, p.tiles_n, tm, tn);
        const int m0 = tm * BM + BMC * (int)rank, n0 = tn * TN + halfn * (int)rank;
        for (int g = 0; g < groups; ++g, ++t) {
          if (lap > 0 && !poll_wait(smem_addr(&done[s]), (lap - 1) & 1u, p.timeout_ns)) {
            if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
            ok = false;
            break;
          }
          if (elect_one()) {
            // both CTAs' loads complete on the even CTA's barrier, which expects all their bytes
            const uint32_t fb = full0 + 8u * (uint32_t)s;
            if (rank == 0) mbar_arrive_expect_tx(smem_addr(&full[s]), bytes);
            const uint32_t a = sbase + (uint32_t)(s * kStageBytes), b = a + kPart;
            tma_load_pair(a, &mapA, fb, p.a_mn ? m0 : g * BK, p.a_mn ? g * BK : m0);
            tma_load_pair(b, &mapB, fb, p.b_mn ? n0 : g * BK, p.b_mn ? g * BK : n0);
          }
          if (++s == kStages) {
            s = 0;
            ++lap;
          }
        }
      }
      // leave only when every copy into shared memory has landed (the odd CTA's warp 1 waits for
      // the products that read its last stages)
      if (rank == 0)
        for (int u = t > kStages ? t - kStages : 0; u < t; ++u)
          if (!poll_wait(smem_addr(&full[u % kStages]), (uint32_t)(u / kStages) & 1u, p.timeout_ns) && lane == 0)
            atomicOr(p.fault, (unsigned)kFaultDrainWait);
    } else if (warp == 1) {
      int t = 0;  // groups whose products have been issued (odd CTA: will be)
      if (rank != 0) {
        t = units;
      } else {
        // ---------------------------------------------- products (even CTA)
        const uint32_t astep = step_of(p.a_mn), bstep = step_of(p.b_mn);
        const uint32_t desc0 = desc_lo(sbase);
        int s = 0, b = 0;
        uint32_t s_lap = 0, b_lap = 0;
        bool ok = poll_wait(smem_addr(&full[0]), 0u, p.timeout_ns);
        while (ok && t < units) {
          ok = b_lap == 0 || poll_wait(smem_addr(&acc_empty[b]), (b_lap - 1) & 1u, p.timeout_ns);
          if (!ok) break;
          tmem_fence_after_sync();
          if (elect_one()) {
            const uint32_t acc = tmem + (uint32_t)(b * TN);
            const uint32_t ad = desc0 + (uint32_t)(s * (kStageBytes >> 4)), bd = ad + (kPart >> 4);
#pragma unroll
            for (uint32_t ks = 0; ks < BK / 32; ++ks)
              mma_f8_pair(acc, make_desc(ad + ks * astep), make_desc(bd + ks * bstep), p.idesc, ks == 0 ? 0u : 1u);
            mma_commit_pair(smem_addr(&done[s]));  // in both CTAs: stage s is free, the accumulator holds group t
          }
          __syncwarp();
          ++t;
          if (++b == bufs) {
            b = 0;
            ++b_lap;
          }
          if (++s == kStages) {
            s = 0;
            ++s_lap;
          }
          // the next group's operands, while this one's products run
          if (t < units) ok = poll_wait(smem_addr(&full[s]), s_lap & 1u, p.timeout_ns);
        }
        if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
      }
      // leave only when every product has completed and its commits have landed in this CTA
      for (int u = t > kStages ? t - kStages : 0; u < t; ++u)
        if (!poll_wait(smem_addr(&done[u % kStages]), (uint32_t)(u / kStages) & 1u, p.timeout_ns)) {
          if (lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
          break;
        }
    } else {
      // ------------------------------------------------ scales, 8 groups at a time, up to kChunks ahead
      // of the folders (the latency of a load is several groups' time): warp 2 of this CTA's 128 rows,
      // warp 3 of the tile's columns or column blocks.
      const uint32_t ring = sbase + (uint32_t)(kStages * kStageBytes + kFoldWarps * kOutBytes);
      int c = 0;
      uint32_t lap = 0;
      bool ok = true;
      for (int i = 0; ok && i < my_tiles; ++i) {
        int tm, tn;
        tile_coords(cl + i * p.clusters, p.tiles_m, p.tiles_n, tm, tn);
        const bool rows = warp == 2;
        const int first = rows ? tm * BM + BMC * (int)rank : tn * TN;
        const int last = (rows ? p.out.M : p.out.N) - 1;
        const Fp8Scales& sc = rows ? p.sa : p.sb;
        const int n = rows ? BMC : COLS ? TN : 3;
        const int pitch = rows ? BMC : Sc::kB;
        for (int g0 = 0; g0 < groups; g0 += kChunk) {
          if (lap > 0 && !poll_wait(smem_addr(&scale_empty[c]), (lap - 1) & 1u, p.timeout_ns)) {
            if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
            ok = false;
            break;
          }
          const uint32_t dst = ring + 4u * (uint32_t)(c * Sc::kFloats + (rows ? 0 : kChunk * BMC));
          const int count = min(kChunk, groups - g0);
          for (int j = lane; j < n; j += 32) {
            const int64_t at = rows || COLS ? min(first + j, last) >> sc.shift : min((first >> 7) + j, last >> 7);
            const int64_t src = at * sc.si + (int64_t)g0 * sc.sk, held = extent(sc, last + 1, groups);
            for (int g = 0; g < count; ++g)
              copy4_async(p.out.guard, kSiteScale, dst + 4u * (uint32_t)(g * pitch + j), sc.p, src + (int64_t)g * sc.sk, held);
          }
          copies_arrive(smem_addr(&scale_full[c]));
          if (OUT != kOutPlain && rows) {  // the rows in equal parts, one with each chunk
            const int chunks = (groups + kChunk - 1) / kChunk, at = g0 / kChunk;
            prefetch_c(p.out, first + BMC * at / chunks, first + BMC * (at + 1) / chunks, tn * TN, TN);
          }
          if (++c == Sc::kChunks) {
            c = 0;
            ++lap;
          }
        }
      }
      copies_wait_all();
    }
  } else {
    more_registers<kFoldRegs>();
    // ------------------------------------------------ folders, then D (both CTAs)
    const int q = warp & 3;                     // TMEM lane quarter this warp may access
    const int part = (warp - kFirstFold) >> 2;  // which half of the tile's columns
    constexpr int cols = TN / 2;
    static_assert(cols % kLoadCols == 0, "whole loads");
    static_assert(cols <= 128 && 128 % cols == 0, "a thread's columns lie in one column block");
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(cols * part);
    uint8_t* out = smem_raw + pad + kStages * kStageBytes + (warp - kFirstFold) * kOutBytes;
    const float* scales = reinterpret_cast<const float*>(smem_raw + pad + kStages * kStageBytes + kFoldWarps * kOutBytes);
    float2 sum[cols / 2];
#pragma unroll
    for (int e = 0; e < cols / 2; ++e) sum[e] = make_float2(0.0f, 0.0f);
    bool ok = true;
    bool seen = false;                      // the group's products were done when last looked at (COLS)
    int s = 0, b = 0, c = 0;                // stage, accumulator and scale chunk of the next group
    uint32_t s_lap = 0, c_lap = 0;
    for (int i = 0; ok && i < my_tiles; ++i) {
      int tm, tn;
      tile_coords(cl + i * p.clusters, p.tiles_m, p.tiles_n, tm, tn);
      const int c0 = tn * TN + cols * part;
      // where this thread's column scales (or its column block's) lie among a group's
      const int b_at = COLS ? cols * part : (c0 >> 7) - ((tn * TN) >> 7);
      for (int g = 0; g < groups; ++g) {
        const int in_chunk = g & (kChunk - 1);
        if (in_chunk == 0) ok = poll_wait(smem_addr(&scale_full[c]), c_lap & 1u, p.timeout_ns);
        if (!COLS || !__all_sync(0xffffffffu, seen)) ok = ok && poll_wait(smem_addr(&done[s]), s_lap & 1u, p.timeout_ns);
        if (!ok) {
          if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
          break;
        }
        tmem_fence_after_sync();
        const uint32_t acc = tq + (uint32_t)(b * TN);
        const float* sc = scales + c * Sc::kFloats;
        const float* scb = sc + kChunk * BMC + in_chunk * Sc::kB + b_at;
        float s0 = 0.0f;
        // 32 columns at a time, the next ones on their way while these are added
        const auto add = [&](auto first, float* v) {
          constexpr int kFirst = decltype(first)::value;
#pragma unroll
          for (int k = 0; k < kLoadCols; k += 8) {
            float* x = v + k;
#pragma unroll
            for (int e = 0; e < 8; ++e) asm volatile("" : "+f"(x[e]));  // used behind the wait only
            float2* m = &sum[(kFirst + k) / 2];
            const float2 w2 = make_float2(s0, s0);
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = __ffma2_rn(make_float2(x[2 * e], x[2 * e + 1]), w2, m[e]);
          }
        };
        const auto load = [&](auto first, float (&v)[kLoadCols]) { tmem_ld(acc + (uint32_t)decltype(first)::value, v); };
        // With a scale per column the fold takes longer than the products: the next group's are then done
        // before this one's last columns are added, and asking beforehand saves the wait's latency (182 to
        // 171 us for 4096 x 4096 x 8192; where the fold waits for the products it costs 4%).
        const auto look = [&] {
          const int ns = s + 1 == kStages ? 0 : s + 1;
          seen = mbar_test(smem_addr(&done[ns]), (s_lap + (ns == 0)) & 1u);
        };
        const auto release = [&] {  // the whole accumulator is in registers: hand it back to the issuer
          tmem_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(smem_addr(&acc_empty[b]), 0);
        };
        constexpr std::integral_constant<int, 0> c_0{};
        constexpr std::integral_constant<int, kLoadCols> c_1{};
        constexpr std::integral_constant<int, 2 * kLoadCols> c_2{};
        constexpr std::integral_constant<int, 3 * kLoadCols> c_3{};
        if constexpr (COLS) {
          // as fragments a lane holds 2 of 8 columns and 4 of 32 rows: 32 column scales to read and not 128
          float va[kLoadCols], vb[kLoadCols];
          float2 wa[kLoadCols / 8], wb[kLoadCols / 8];
          float rs[4];
          const auto fetch = [&](auto first, float* v, float2* w) {
            constexpr int kFirst = decltype(first)::value;
            tmem_ld_fragments(acc + (uint32_t)kFirst, v);
            tmem_ld_fragments(acc + (uint32_t)kFirst + (16u << 16), v + kLoadCols / 2);
#pragma unroll
            for (int j = 0; j < kLoadCols / 8; ++j)
              w[j] = *reinterpret_cast<const float2*>(scb + kFirst + 8 * j + 2 * (lane & 3));
          };
          const auto scaled = [&](auto first, float* v, const float2* w) {
            constexpr int kFirst = decltype(first)::value;
#pragma unroll
            for (int e = 0; e < kLoadCols; ++e) asm volatile("" : "+f"(v[e]));  // used behind the wait only
#pragma unroll
            for (int j = 0; j < kLoadCols / 8; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // rows lane / 4 + 8 k
                const float* x = v + (k / 2) * (kLoadCols / 2) + 4 * j + 2 * (k % 2);
                float2& m = sum[kFirst / 2 + 4 * j + k];
                // the two scales first: either alone may be far from 1
                m = __ffma2_rn(make_float2(x[0], x[1]), __fmul2_rn(w[j], make_float2(rs[k], rs[k])), m);
              }
          };
          fetch(c_0, va, wa);
#pragma unroll
          for (int k = 0; k < 4; ++k) rs[k] = sc[in_chunk * BMC + 32 * q + (lane >> 2) + 8 * k];
          tmem_wait_ld();
          if constexpr (cols > c_1) fetch(c_1, vb, wb);
          else release();
          scaled(c_0, va, wa);
          if constexpr (cols > c_1) {
            tmem_wait_ld();
            if constexpr (cols > c_2) fetch(c_2, va, wa);
            else release();
            scaled(c_1, vb, wb);
          }
          if constexpr (cols > c_2) {
            tmem_wait_ld();
            fetch(c_3, vb, wb);
            scaled(c_2, va, wa);
            tmem_wait_ld();
            release();
            look();
            scaled(c_3, vb, wb);
          }
        } else {
          float va[kLoadCols], vb[kLoadCols];
          load(c_0, va);
          s0 = sc[in_chunk * BMC + 32 * q + lane] * scb[0];
          tmem_wait_ld();
          if constexpr (cols > c_1) load(c_1, vb);
          else release();
          add(c_0, va);
          if constexpr (cols > c_1) {
            tmem_wait_ld();
            if constexpr (cols > c_2) load(c_2, va);
            else release();
            add(c_1, vb);
          }
          if constexpr (cols > c_2) {
            tmem_wait_ld();
            if constexpr (cols > c_3) load(c_3, vb);
            else release();
            add(c_2, va);
          }
          if constexpr (cols > c_3) {
            tmem_wait_ld();
            release();
            add(c_3, vb);
          }
        }
        if (in_chunk == kChunk - 1 || g == groups - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&scale_empty[c]));
          if (++c == Sc::kChunks) {
            c = 0;
            ++c_lap;
          }
        }
        if (++b == bufs) b = 0;
        if (++s == kStages) {
          s = 0;
          ++s_lap;
        }
      }
      // This thread holds columns c0 .. c0 + cols - 1 of its row; 32 rows x 32 columns at a time go
      // through shared memory.
      const int row0 = tm * BM + BMC * (int)rank + 32 * q;
      if (ok && OUT == kOutPlain) {
        // in D's type and the order TMA reads, which writes the piece (as far as it is in D) by itself
        if (p.out.bf16) tma_out<true, COLS>(mapD, out, p.out, row0, c0, sum);
        else            tma_out<false, COLS>(mapD, out, p.out, row0, c0, sum);
      } else if (ok) {
        constexpr int pitch = COLS ? kOutPitchFragments : kOutPitch;
        float* piece = reinterpret_cast<float*>(out);
#pragma unroll
        for (int at = 0; at < cols; at += 32) {
          __syncwarp();
          if constexpr (COLS) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              *reinterpret_cast<float2*>(piece + ((lane >> 2) + 8 * (e % 4)) * pitch + 8 * (e / 4) + 2 * (lane & 3)) =
                  sum[at / 2 + e];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(piece + lane * pitch + 4 * e) =
                  make_float4(sum[at / 2 + 2 * e].x, sum[at / 2 + 2 * e].y, sum[at / 2 + 2 * e + 1].x,
                              sum[at / 2 + 2 * e + 1].y);
          }
          __syncwarp();
          store_piece<OUT>(p.out, row0, c0 + at, piece, pitch);
        }
      }
#pragma unroll
      for (int e = 0; e < cols / 2; ++e) sum[e] = make_float2(0.0f, 0.0f);
    }
    if (OUT == kOutPlain && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  tmem_fence_before_sync();
  __syncthreads();
  // Bounded handshake of the two CTAs: neither releases its TMEM or exits while the other may
  // still arrive on its barriers or have products read its shared memory and TMEM.
  if (threadIdx.x == 0) {
    mbar_arrive_remote(smem_addr(&fin), rank ^ 1u);
    if (!mbar_wait(smem_addr(&fin), 0u, p.timeout_ns)) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  }
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

}  // namespace
}  // namespace f8

namespace f8 {
namespace {
// f(kernel, its dynamic shared memory) for the kernel of a tile width and scale form.
template <int OUT, typename F>
cudaError_t with_pair_kernel(int tile_n, bool cols, const F& f) {
  constexpr size_t kBlocks = ScaleCfg<false>::kSmem, kCols = ScaleCfg<true>::kSmem;
  switch (tile_n) {
    case 256: return cols ? f(fp8_pair_kernel<256, true, OUT>, kCols) : f(fp8_pair_kernel<256, false, OUT>, kBlocks);
    case 128: return cols ? f(fp8_pair_kernel<128, true, OUT>, kCols) : f(fp8_pair_kernel<128, false, OUT>, kBlocks);
    case 64: return cols ? f(fp8_pair_kernel<64, true, OUT>, kCols) : f(fp8_pair_kernel<64, false, OUT>, kBlocks);
  }
  return cudaErrorInvalidValue;
}

template <int OUT>
cudaError_t prepare_pair() {
  for (int tile_n : kFp8PairTiles)
    for (int cols = 0; cols < 2; ++cols) {
      const cudaError_t e = with_pair_kernel<OUT>(tile_n, cols != 0, [](auto kernel, size_t smem) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      });
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

template <int OUT>
cudaError_t launch_pair(int tile_n, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapD,
                        const Fp8PairParams& p, cudaStream_t stream) {
  return with_pair_kernel<OUT>(tile_n, p.sb.shift == 0, [&](auto kernel, size_t smem) {
    kernel<<<2u * (unsigned)p.clusters, kThreads, smem, stream>>>(mapA, mapB, mapD, p);
    return cudaGetLastError();
  });
}
}  // namespace
}  // namespace f8

#define SGEMM_DEFINE_FP8_PAIR(name, OUT)                                                                       \
  cudaError_t prepare_fp8_pair_##name() { return f8::prepare_pair<OUT>(); }                                    \
  cudaError_t launch_fp8_pair_##name(int tile_n, const CUtensorMap& mapA, const CUtensorMap& mapB,             \
                                     const CUtensorMap& mapD, const Fp8PairParams& p, cudaStream_t stream) {   \
    return f8::launch_pair<OUT>(tile_n, mapA, mapB, mapD, p, stream);                                          \
  }

}  // namespace sgemm_impl
