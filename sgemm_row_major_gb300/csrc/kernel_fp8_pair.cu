// kernel_fp8_pair.cu -- block-scaled 8-bit product on CTA pairs for sm_103a.
//
//     D = alpha * sum_g sA(i, g) sB(g, j) P_g(i, j) + beta * C,   P_g = sum over 128 k of code products
//
// Clusters of two CTAs on one TPC compute 256 x tile_n tiles (tile_n <= 256, a multiple of 32) with
// tcgen05.mma.cta_group::2.kind::f8f6f4, M = 256, N = tile_n, K = 32, both operands from shared
// memory: each CTA holds 128 rows of A and half of the tile's columns of B.  Four such steps make
// one P_g in a fresh TMEM accumulator (two of 256 columns alternate); 8 warps per CTA read it back
// and add sA sB P_g to sums in FP32 registers, so every scale is an FP32 number and no sum is held
// in fewer bits.  At tile_n = 256 the tensor cores need 512 cycles for a group and the folders 256
// cycles of the FMA pipes, so the fold is hidden behind the products.
//
// Either operand may be stored along K or across it: the tensor core reads both orders, so a
// gradient's product takes the weights and activations as the forward pass left them.
//
// Warp 0 loads (TMA, 6 stages of 32 KB), warp 1 of the even CTA issues the products, warps 2-9 fold
// and write D.  Persistent clusters take tiles round robin in an order that keeps 8 rows of tiles
// together (their A and B panels stay in L2); tile_n is chosen by the caller so that the last round
// of tiles is nearly full.
#include "fp8_gemm.cuh"

namespace sgemm_impl {
namespace f8 {
namespace {

using namespace tc;

constexpr int BM = 256, BMC = 128, BK = 128;
constexpr int kPart = 128 * BK;           // 16 KB: one operand's tile in one CTA
constexpr int kStageBytes = 2 * kPart;
constexpr int kStages = 6;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
constexpr int kFoldWarps = 8;
constexpr int kThreads = 32 * (2 + kFoldWarps);
constexpr int kAccBufs = 2;
constexpr uint32_t kAccCols = 256;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxHalf = 128;             // accumulator columns a folder thread owns at most

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster,
                                              int32_t inner, int32_t outer) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(inner), "r"(outer), "r"(0)
      : "memory");
}

// The 128 threads of the four warps that share a half of the accumulator's columns.
__device__ __forceinline__ void half_barrier(int half) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
}

// COLS: B has one scale per column (weight gradients), else one per 128 columns.
template <bool COLS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                    const __grid_constant__ Fp8PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
  __shared__ __align__(8) uint64_t acc_full[kAccBufs], acc_empty[kAccBufs];
  __shared__ __align__(8) uint64_t fin;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float col_scale[COLS ? 2 : 1][2][COLS ? kMaxHalf : 1];

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t sbase = raw_addr + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cl = (int)cluster_id_x();
  const int groups = (p.K + BK - 1) / BK;
  const int tiles = p.tiles_m * p.tiles_n;
  const int my_tiles = cl < tiles ? (tiles - cl + p.clusters - 1) / p.clusters : 0;
  const int units = my_tiles * groups;
  const int halfn = p.tile_n / 2;  // columns of B this CTA loads, and accumulator columns of a folder

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    for (int b = 0; b < kAccBufs; ++b) {
      mbar_init(smem_addr(&acc_full[b]), 1);
      mbar_init(smem_addr(&acc_empty[b]), 2 * kFoldWarps);
    }
    mbar_init(smem_addr(&fin), 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_addr(&tmem_slot), kTmemCols);
  tmem_fence_before_sync();
  cluster_sync();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------ loads (each CTA: its rows of A, its columns of B)
    if (lane == 0) {
      prefetch_tensormap(&mapA);
      prefetch_tensormap(&mapB);
      const uint32_t bytes = 2u * (uint32_t)(kPart + (p.b_mn ? kPart : halfn * BK));  // both CTAs'
      int t = 0;
      bool ok = true;
      for (int i = 0; ok && i < my_tiles; ++i) {
        int tm, tn;
        tile_coords(cl + i * p.clusters, p.tiles_m, p.tiles_n, tm, tn);
        const int m0 = tm * BM + BMC * (int)rank, n0 = tn * p.tile_n + halfn * (int)rank;
        for (int g = 0; g < groups; ++g, ++t) {
          const int s = t % kStages;
          if (t >= kStages && !mbar_wait(smem_addr(&empty[s]), (uint32_t)((t / kStages) - 1) & 1u, p.timeout_ns)) {
            atomicOr(p.fault, (unsigned)kFaultEmptyWait);
            ok = false;
            break;
          }
          // both CTAs' loads complete on the even CTA's barrier, which expects all their bytes
          const uint32_t fb = map_to_rank(smem_addr(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(smem_addr(&full[s]), bytes);
          const uint32_t a = sbase + (uint32_t)(s * kStageBytes), b = a + kPart;
          tma_load_pair(a, &mapA, fb, p.a_mn ? m0 : g * BK, p.a_mn ? g * BK : m0);
          tma_load_pair(b, &mapB, fb, p.b_mn ? n0 : g * BK, p.b_mn ? g * BK : n0);
        }
      }
      // leave only when every copy into shared memory has landed (the odd CTA's warp 1 waits for
      // the products that read its last stages)
      if (rank == 0)
        for (int u = t > kStages ? t - kStages : 0; u < t; ++u)
          if (!mbar_wait(smem_addr(&full[u % kStages]), (uint32_t)(u / kStages) & 1u, p.timeout_ns))
            atomicOr(p.fault, (unsigned)kFaultDrainWait);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank != 0) {
      bool ok = true;
      for (int u = units > kStages ? units - kStages : 0; ok && u < units; ++u)
        ok = mbar_wait(smem_addr(&empty[u % kStages]), (uint32_t)(u / kStages) & 1u, p.timeout_ns);
      if (!ok) atomicOr(p.fault, (unsigned)kFaultFullWait);
    } else if (lane == 0) {
      // ---------------------------------------------- products (even CTA)
      const uint64_t astep = step_of(p.a_mn), bstep = step_of(p.b_mn);
      int t_done = -1;
      bool ok = true;
      for (int t = 0; ok && t < units; ++t) {
        const int s = t % kStages, b = t % kAccBufs;
        ok = (t < kAccBufs ||
              mbar_wait(smem_addr(&acc_empty[b]), (uint32_t)((t / kAccBufs) - 1) & 1u, p.timeout_ns)) &&
             mbar_wait(smem_addr(&full[s]), (uint32_t)(t / kStages) & 1u, p.timeout_ns);
        if (!ok) break;
        tmem_fence_after_sync();
        const uint32_t acc = tmem + (uint32_t)b * kAccCols;
        const uint32_t a = sbase + (uint32_t)(s * kStageBytes);
        const uint64_t ad = tile_desc(a), bd = tile_desc(a + kPart);
#pragma unroll
        for (int ks = 0; ks < BK / 32; ++ks)
          mma_f8_pair(acc, ad + (uint64_t)ks * astep, bd + (uint64_t)ks * bstep, p.idesc, ks == 0 ? 0u : 1u);
        mma_commit_pair(smem_addr(&empty[s]));     // stage s reusable in both CTAs
        mma_commit_pair(smem_addr(&acc_full[b]));  // accumulator b (both CTAs) holds group t
        t_done = t;
      }
      if (!ok) atomicOr(p.fault, (unsigned)kFaultFullWait);
      // leave only when every product has completed and its commits have landed here
      for (int u = t_done + 1 > kStages ? t_done + 1 - kStages : 0; u <= t_done; ++u)
        if (!mbar_wait(smem_addr(&empty[u % kStages]), (uint32_t)(u / kStages) & 1u, p.timeout_ns))
          atomicOr(p.fault, (unsigned)kFaultDrainWait);
      if (t_done >= 0 &&
          !mbar_wait(smem_addr(&acc_full[t_done % kAccBufs]), (uint32_t)(t_done / kAccBufs) & 1u, p.timeout_ns))
        atomicOr(p.fault, (unsigned)kFaultDrainWait);
    }
  } else {
    // ------------------------------------------------ folders, then D (both CTAs)
    const int q = warp & 3;            // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // which half of the tile's columns
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(halfn * half);
    const int hid = 32 * ((warp - 2) & 3) + lane;  // thread of its half
    float2 sum[kMaxHalf / 2];
#pragma unroll
    for (int e = 0; e < kMaxHalf / 2; ++e) sum[e] = make_float2(0.0f, 0.0f);
    bool ok = true;
    int t = 0;
    for (int i = 0; i < my_tiles; ++i) {
      int tm, tn;
      tile_coords(cl + i * p.clusters, p.tiles_m, p.tiles_n, tm, tn);
      const int row = tm * BM + BMC * (int)rank + 32 * q + lane;
      const int c0 = tn * p.tile_n + halfn * half;
      // scales: this row's, and either the (at most two) column blocks' of this half or one column
      // per thread of the half; the next group's are loaded while this group is waited for
      const float* sa = p.sa.p + (int64_t)(min(row, p.out.M - 1) >> p.sa.shift) * p.sa.si;
      const float *sb0, *sb1;
      const int edge = ((c0 >> 7) + 1) * 128 - c0;  // columns of this half in its first column block
      if (COLS) {
        sb0 = sb1 = p.sb.p + (int64_t)min(c0 + min(hid, halfn - 1), p.out.N - 1) * p.sb.si;
      } else {
        sb0 = p.sb.p + (int64_t)(min(c0, p.out.N - 1) >> 7) * p.sb.si;
        sb1 = p.sb.p + (int64_t)(min(c0 + halfn - 1, p.out.N - 1) >> 7) * p.sb.si;
      }
      float a_next = __ldg(sa), b0_next = __ldg(sb0), b1_next = COLS ? 0.0f : __ldg(sb1);
      for (int g = 0; g < groups; ++g, ++t) {
        const float a_cur = a_next, b0_cur = b0_next, b1_cur = b1_next;
        if (g + 1 < groups) {
          a_next = __ldg(sa + (int64_t)(g + 1) * p.sa.sk);
          b0_next = __ldg(sb0 + (int64_t)(g + 1) * p.sb.sk);
          if (!COLS) b1_next = __ldg(sb1 + (int64_t)(g + 1) * p.sb.sk);
        }
        if (COLS) {  // written two groups ago at the latest read: one barrier per group suffices
          col_scale[t & 1][half][hid] = b0_cur;
          half_barrier(half);
        }
        const int b = t % kAccBufs;
        if (ok) {  // a warp that gave up keeps meeting the others at the barrier
          ok = warp_wait(smem_addr(&acc_full[b]), (uint32_t)(t / kAccBufs) & 1u, p.timeout_ns);
          if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        }
        if (!ok) continue;
        tmem_fence_after_sync();
        const float s0 = a_cur * b0_cur, s1 = a_cur * b1_cur;
#pragma unroll
        for (int ch = 0; ch < kMaxHalf / 32; ++ch) {
          if (32 * ch < halfn) {
            float v[2][16];
            tmem_ld16(tq + (uint32_t)b * kAccCols + (uint32_t)(32 * ch), v[0]);
            if (32 * ch + 16 < halfn) tmem_ld16(tq + (uint32_t)b * kAccCols + (uint32_t)(32 * ch + 16), v[1]);
            tmem_wait_ld();
            if (32 * (ch + 1) >= halfn) {
              // the whole accumulator is in registers: hand it back to the issuer
              tmem_fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive_remote(smem_addr(&acc_empty[b]), 0);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (32 * ch + 16 * c >= halfn) continue;
              tmem_ld_ready(v[c]);
              if (COLS) {
                const float4* cs = reinterpret_cast<const float4*>(&col_scale[t & 1][half][COLS ? 32 * ch + 16 * c : 0]);
                const float2 sa2 = make_float2(a_cur, a_cur);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float4 w = cs[e];
                  float2& m0 = sum[(32 * ch + 16 * c) / 2 + 2 * e];
                  float2& m1 = sum[(32 * ch + 16 * c) / 2 + 2 * e + 1];
                  m0 = __ffma2_rn(__fmul2_rn(make_float2(v[c][4 * e], v[c][4 * e + 1]), make_float2(w.x, w.y)), sa2, m0);
                  m1 = __ffma2_rn(__fmul2_rn(make_float2(v[c][4 * e + 2], v[c][4 * e + 3]), make_float2(w.z, w.w)), sa2, m1);
                }
              } else {
                const float s = 32 * ch + 16 * c < edge ? s0 : s1;
                const float2 s2 = make_float2(s, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  float2& m = sum[(32 * ch + 16 * c) / 2 + e];
                  m = __ffma2_rn(make_float2(v[c][2 * e], v[c][2 * e + 1]), s2, m);
                }
              }
            }
          }
        }
      }
      // this thread holds columns c0 .. c0 + halfn - 1 of its row
      if (ok && row < p.out.M) {
#pragma unroll
        for (int e = 0; e < kMaxHalf / 8; ++e) {
          const int col = c0 + 8 * e;
          if (8 * e >= halfn || col >= p.out.N) continue;
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] = sum[4 * e + k].x;
            v[2 * k + 1] = sum[4 * e + k].y;
          }
          if (p.out.vec && col + 8 <= p.out.N) {
            store_eight(p.out, row, col, v);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (col + k < p.out.N) store_one(p.out, row, col + k, v[k]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kMaxHalf / 2; ++e) sum[e] = make_float2(0.0f, 0.0f);
    }
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

cudaError_t prepare_fp8_pair() {
  cudaError_t e = cudaFuncSetAttribute(f8::fp8_pair_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       f8::kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(f8::fp8_pair_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, f8::kSmemBytes);
  return e;
}

cudaError_t launch_fp8_pair(const CUtensorMap& mapA, const CUtensorMap& mapB, const Fp8PairParams& p,
                            cudaStream_t stream) {
  const dim3 grid(2u * (unsigned)p.clusters);
  if (p.sb.shift == 0) f8::fp8_pair_kernel<true><<<grid, f8::kThreads, f8::kSmemBytes, stream>>>(mapA, mapB, p);
  else f8::fp8_pair_kernel<false><<<grid, f8::kThreads, f8::kSmemBytes, stream>>>(mapA, mapB, p);
  return cudaGetLastError();
}

}  // namespace sgemm_impl
