// kernel_fp8_short.cu -- block-scaled 8-bit product with a short side, for sm_103a; and the small
// passes around the products (aligned copies of codes, D = beta * C).
//
// The same sum as kernel_fp8_pair.cuh for products whose time is that of reading the long operand
// (the weights of a decoding step).  The long side runs along the 128 rows of the tensor core, the
// short one along its columns (tile_s <= 128, a multiple of 16), so a row of one token costs a
// 128 x 16 tile and not a 256-row one; when the short side is M the tile is D transposed and is
// written along the long side all the same.  One CTA per tile and K share: a cluster of `split`
// CTAs (1, 2, 4 or 8) divides the groups of 128 k of a tile, each folds its groups into FP32 sums
// as the pair kernel does, leaves them in shared memory, and the cluster adds the shares in rank
// order, each CTA a part of the tile read from its peers' shared memory: no workspace, one launch,
// and the same result every time.
//
// Warp 0 loads (TMA; as many stages as fit twice per SM), warp 1 issues the products, warps 2-5 fold.
#include "fp8_gemm.cuh"

namespace sgemm_impl {
namespace f8 {
namespace {

using namespace tc;

constexpr int BL = 128, BK = 128;
constexpr int kFoldThreads = 128;
constexpr int kThreads = 64 + kFoldThreads;
constexpr int kMaxStages = 12;
constexpr int kMaxS = 128;
constexpr int kMaxSmem = 220 * 1024;
constexpr int kPitch = BL + 1;  // words between the columns of a share: lanes along rows or columns both hit 32 banks

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t inner,
                                         int32_t outer) {
  tma_load_3d(dst, map, bar, inner, outer, 0);
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void fold_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// MAXS: the largest tile_s this form holds sums for (32 columns leave registers for more CTAs).
template <int MAXS>
__global__ void __launch_bounds__(kThreads, 2) fp8_short_kernel(const __grid_constant__ CUtensorMap mapL,
                                                                const __grid_constant__ CUtensorMap mapS,
                                                                const __grid_constant__ Fp8ShortParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float col_scale[2][kMaxS];

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  float* share = reinterpret_cast<float*>(smem_raw + pad);  // over the ring, once it is drained
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % p.split;  // of the cluster: blocks of a cluster are consecutive
  const int tile = (int)blockIdx.x / p.split;
  const int l0 = (tile / p.tiles_s) * BL, s0 = (tile % p.tiles_s) * p.tile_s;
  const int groups = (p.K + BK - 1) / BK;
  const int g0 = (int)((int64_t)groups * rank / p.split), g1 = (int)((int64_t)groups * (rank + 1) / p.split);
  const int units = g1 - g0;
  const uint32_t tmem_cols = p.tile_s <= 32 ? 64u : p.tile_s <= 64 ? 128u : 256u;  // two accumulators

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&acc_full[b]), 1);
      mbar_init(smem_addr(&acc_empty[b]), kFoldThreads / 32);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), tmem_cols);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const uint32_t acc_step = tmem_cols / 2;

  if (warp == 0) {
    // ------------------------------------------------ loads
    const uint32_t bytes = (uint32_t)(BL * BK + (p.s_mn ? 128 * BK : p.tile_s * BK));
    int t = 0, s = 0;
    uint32_t lap = 0;
    for (; t < units; ++t) {
      if (lap > 0 && !poll_wait(smem_addr(&empty[s]), (lap - 1) & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
        break;
      }
      if (elect_one()) {
        const int k0 = (g0 + t) * BK;
        const uint32_t bar = smem_addr(&full[s]), a = sbase + (uint32_t)(s * p.stage_bytes);
        mbar_arrive_expect_tx(bar, bytes);
        tma_load(a, &mapL, bar, p.l_mn ? l0 : k0, p.l_mn ? k0 : l0);
        tma_load(a + BL * BK, &mapS, bar, p.s_mn ? s0 : k0, p.s_mn ? k0 : s0);
      }
      if (++s == p.stages) {
        s = 0;
        ++lap;
      }
    }
    // leave only when every copy into shared memory has landed
    for (int u = t > p.stages ? t - p.stages : 0; u < t; ++u)
      if (!poll_wait(smem_addr(&full[u % p.stages]), (uint32_t)(u / p.stages) & 1u, p.timeout_ns) && lane == 0)
        atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else if (warp == 1) {
    // ------------------------------------------------ products
    const uint32_t lstep = step_of(p.l_mn), sstep = step_of(p.s_mn);
    int t = 0, s = 0;
    uint32_t lap = 0;
    for (; t < units; ++t) {
      const int b = t & 1;
      if ((t >= 2 && !poll_wait(smem_addr(&acc_empty[b]), (uint32_t)((t / 2) - 1) & 1u, p.timeout_ns)) ||
          !poll_wait(smem_addr(&full[s]), lap & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        break;
      }
      tmem_fence_after_sync();
      if (elect_one()) {
        const uint32_t a = sbase + (uint32_t)(s * p.stage_bytes);
        const uint32_t ld = desc_lo(a), sd = desc_lo(a + BL * BK);
#pragma unroll
        for (int ks = 0; ks < BK / 32; ++ks)
          mma_f8(tmem + (uint32_t)b * acc_step, make_desc(ld + (uint32_t)ks * lstep),
                 make_desc(sd + (uint32_t)ks * sstep), p.idesc,
                 ks == 0 ? 0u : 1u);
        mma_commit(smem_addr(&empty[s]));
        mma_commit(smem_addr(&acc_full[b]));
      }
      __syncwarp();
      if (++s == p.stages) {
        s = 0;
        ++lap;
      }
    }
    // leave only when every product has completed and its commits have landed
    bool ok = true;
    for (int u = t > p.stages ? t - p.stages : 0; u < t; ++u)
      ok = ok && poll_wait(smem_addr(&empty[u % p.stages]), (uint32_t)(u / p.stages) & 1u, p.timeout_ns);
    for (int u = t > 2 ? t - 2 : 0; u < t; ++u)
      ok = ok && poll_wait(smem_addr(&acc_full[u & 1]), (uint32_t)(u / 2) & 1u, p.timeout_ns);
    if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  }

  // ------------------------------------------------ folders: row 32q + lane of the tile, all its columns
  float2 sum[MAXS / 2];
  const int row = 32 * (warp & 3) + lane;  // warps 2, 3, 4, 5: TMEM lane quarters 2, 3, 0, 1
  bool ok = true;
  if (warp >= 2) {
    const int q = warp & 3;
    const int fid = (int)threadIdx.x - 64;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
#pragma unroll
    for (int e = 0; e < MAXS / 2; ++e) sum[e] = make_float2(0.0f, 0.0f);
    const float* sl = p.sl.p + (int64_t)(min(l0 + row, p.L - 1) >> p.sl.shift) * p.sl.si + (int64_t)g0 * p.sl.sk;
    const float* ss = p.ss.p + (int64_t)(min(s0 + min(fid, p.tile_s - 1), p.S - 1) >> p.ss.shift) * p.ss.si +
                      (int64_t)g0 * p.ss.sk;
    float l_next = units > 0 ? __ldg(sl) : 0.0f, s_next = units > 0 ? __ldg(ss) : 0.0f;
    for (int t = 0; t < units; ++t) {
      const int b = t & 1;
      const float l_cur = l_next;
      col_scale[b][fid] = s_next;  // last read two groups ago: one barrier per group suffices
      if (t + 1 < units) {
        l_next = __ldg(sl + (int64_t)(t + 1) * p.sl.sk);
        s_next = __ldg(ss + (int64_t)(t + 1) * p.ss.sk);
      }
      fold_barrier();
      if (ok) {  // a warp that gave up keeps meeting the others at the barrier
        ok = poll_wait(smem_addr(&acc_full[b]), (uint32_t)(t / 2) & 1u, p.timeout_ns);
        if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
      }
      if (!ok) continue;
      tmem_fence_after_sync();
      const float2 l2 = make_float2(l_cur, l_cur);
#pragma unroll
      for (int c = 0; c < MAXS / 16; ++c) {
        if (16 * c < p.tile_s) {
          float v[16];
          tmem_ld16(tq + (uint32_t)b * acc_step + (uint32_t)(16 * c), v);
          tmem_wait_ld();
          if (16 * (c + 1) >= p.tile_s) {
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&acc_empty[b]));
          }
          tmem_ld_ready(v);
          const float4* cs = reinterpret_cast<const float4*>(&col_scale[b][16 * c]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 w = cs[e];
            float2& m0 = sum[8 * c + 2 * e];
            float2& m1 = sum[8 * c + 2 * e + 1];
            m0 = __ffma2_rn(__fmul2_rn(make_float2(v[4 * e], v[4 * e + 1]), make_float2(w.x, w.y)), l2, m0);
            m1 = __ffma2_rn(__fmul2_rn(make_float2(v[4 * e + 2], v[4 * e + 3]), make_float2(w.z, w.w)), l2, m1);
          }
        }
      }
    }
  }

  // ------------------------------------------------ the shares, added in rank order
  tmem_fence_before_sync();
  __syncthreads();  // the ring is drained: loads have landed and the products that read it are done
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, tmem_cols);
  if (warp >= 2) {
#pragma unroll
    for (int c = 0; c < MAXS / 16; ++c)
      if (16 * c < p.tile_s)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          share[(16 * c + 2 * e) * kPitch + row] = sum[8 * c + e].x;
          share[(16 * c + 2 * e + 1) * kPitch + row] = sum[8 * c + e].y;
        }
  }
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  // this CTA's part of the tile: its share of the columns (D transposed: lanes along the long side)
  // or of the rows (lanes along the short side, the columns of D)
  const int nl = min(BL, p.L - l0), ns = min(p.tile_s, p.S - s0);
  const uint32_t share_addr = sbase;
  const int parts = p.trans ? ns : nl;
  const int b0 = parts * rank / p.split, b1 = parts * (rank + 1) / p.split;
  const int inner = p.trans ? nl : ns;
  for (int i = (int)threadIdx.x; i < (b1 - b0) * inner; i += kThreads) {
    const int outer_i = b0 + i / inner, inner_i = i % inner;
    const int l = p.trans ? inner_i : outer_i, s = p.trans ? outer_i : inner_i;
    const uint32_t at = share_addr + 4u * (uint32_t)(s * kPitch + l);
    float v = 0.0f;
    if (p.split == 1) {
      v = share[s * kPitch + l];
    } else {
      float u[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < p.split) u[r] = ld_cluster(map_to_rank(at, (uint32_t)r));
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < p.split) v += u[r];
    }
    if (p.trans) store_one(p.out, s0 + s, l0 + l, v);
    else         store_one(p.out, l0 + l, s0 + s, v);
  }
  if (p.split > 1) {
    __syncthreads();
    cluster_sync();  // no CTA leaves while a peer may read its share
  }
}

__global__ void __launch_bounds__(256) repack_kernel(const uint8_t* __restrict__ src, int64_t ld, int64_t rows,
                                                     int64_t cols, uint8_t* __restrict__ dst, int64_t ldd) {
  const int64_t chunks = ldd / 16, total = rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / chunks, c = (i - r * chunks) * 16;
    const uint8_t* s = src + r * ld + c;
    const int n = (int)min((int64_t)16, cols - c);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k < n) w[k / 4] |= (uint32_t)s[k] << (8 * (k % 4));
    *reinterpret_cast<uint4*>(dst + r * ldd + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__global__ void __launch_bounds__(256) scale_kernel(const Fp8Out o) {
  const int64_t total = (int64_t)o.M * o.N;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / o.N, col = i - row * o.N;
    const float x = o.beta == 0.0f ? 0.0f : o.beta * read_c(o, row * o.ldc + col);
    const int64_t d = row * o.ldd + col;
    if (o.bf16) static_cast<__nv_bfloat16*>(o.D)[d] = __float2bfloat16_rn(x);
    else        static_cast<float*>(o.D)[d] = x;
  }
}

}  // namespace
}  // namespace f8

size_t fp8_short_smem(int tile_s, int stages, int stage_bytes) {
  const size_t ring = (size_t)stages * stage_bytes, share = (size_t)tile_s * f8::kPitch * 4;
  return (ring > share ? ring : share) + 1024;
}

cudaError_t prepare_fp8_short() {
  cudaError_t e = cudaFuncSetAttribute(f8::fp8_short_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       f8::kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(f8::fp8_short_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, f8::kMaxSmem);
  return e;
}

cudaError_t launch_fp8_short(const CUtensorMap& mapL, const CUtensorMap& mapS, const Fp8ShortParams& p,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tiles_l * p.tiles_s * p.split));
  cfg.blockDim = dim3(f8::kThreads);
  cfg.dynamicSmemBytes = fp8_short_smem(p.tile_s, p.stages, p.stage_bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.tile_s <= 32 ? cudaLaunchKernelEx(&cfg, f8::fp8_short_kernel<32>, mapL, mapS, p)
                        : cudaLaunchKernelEx(&cfg, f8::fp8_short_kernel<128>, mapL, mapS, p);
}

cudaError_t launch_fp8_repack(const void* src, int64_t ld, int64_t rows, int64_t cols, void* dst, int64_t ldd,
                              cudaStream_t stream) {
  const int64_t blocks = (rows * (ldd / 16) + 255) / 256;
  f8::repack_kernel<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(
      static_cast<const uint8_t*>(src), ld, rows, cols, static_cast<uint8_t*>(dst), ldd);
  return cudaGetLastError();
}

cudaError_t launch_fp8_scale(const Fp8Out& o, cudaStream_t stream) {
  const int64_t blocks = ((int64_t)o.M * o.N + 255) / 256;
  f8::scale_kernel<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(o);
  return cudaGetLastError();
}

}  // namespace sgemm_impl
