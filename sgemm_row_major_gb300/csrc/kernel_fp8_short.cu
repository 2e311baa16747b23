// kernel_fp8_short.cu -- block-scaled 8-bit product with a short side, for sm_103a; and the small
// passes around the products (aligned copies of codes, D = beta * C).
//
// The same sum as kernel_fp8_pair.cuh for products whose time is that of reading the long operand
// (the weights of a decoding step).  The long side runs along the 128 rows of the tensor core, the
// short one along its columns (tile_s 16, 32, 64 or 128), so a row of one token costs a
// 128 x 16 tile and not a 256-row one; when the short side is M the tile is D transposed and is
// written along the long side all the same.  One CTA per tile and K share: a cluster of `split`
// CTAs (1, 2, 4 or 8) divides the groups of 128 k of a tile, each folds its groups into FP32 sums
// as the pair kernel does, leaves them in shared memory, and the cluster adds the shares in rank
// order, each CTA a part of the tile read from its peers' shared memory: no workspace, one launch,
// and the same result every time.
//
// Warp 0 loads (TMA), warp 1 issues the products, warp 2 loads scales a chunk of 8 groups ahead, warps
// 4-7 fold.  tile_s is a template argument (16, 32, 64 or 128): the fold's branches cost as much as its
// work otherwise.  Two CTAs per SM share its memory (one at 128 columns, whose sums need the registers).
//
// What bounds it: a stream of the long operand, but a CTA starts, folds and joins in 4 us and takes 310 ns
// (16 columns) to 545 ns (128) for a group, where its 16 KB are 370 ns of an SM's share of the memory's
// bandwidth: 1 x 4096 x 4096 (17 MB) 7.0 us, 64 x 4096 x 16384 (68 MB) 19.1 us, 3.6 TB/s.  More shares
// shorten the groups' part and lengthen the joining.
#include "fp8_gemm.cuh"

namespace sgemm_impl {
namespace f8 {
namespace {

using namespace tc;

constexpr int BL = 128, BK = 128;
constexpr int kFirstFold = 4, kFoldWarps = 4;
constexpr int kThreads = 32 * (kFirstFold + kFoldWarps);
constexpr int kMaxStages = kFp8ShortMaxStages;
static_assert(kThreads == kFp8ShortThreads, "the plan's figure");
constexpr int kMaxSmem = 220 * 1024;
// A share lies in shared memory in the order in which it is read, along the long side (D transposed) or
// the short one: peers' reads of 32 consecutive words are one access, at any other step 32 (a product of
// 1000 x 300 x 900 took 25 us and not 8).  The odd pitch keeps the folders' writes free of conflicts.
__host__ __device__ constexpr int share_pitch(bool trans, int tile_s) { return trans ? BL + 1 : tile_s + 1; }
__host__ __device__ constexpr int share_words(int tile_s) { return BL * tile_s + (BL > tile_s ? BL : tile_s); }
constexpr int kChunkGroups = 8;  // groups whose scales are loaded together
constexpr int kChunks = 2;       // in shared memory

__host__ __device__ constexpr int chunk_floats(int tile_s) { return kChunkGroups * (BL + tile_s); }

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int TS>
__global__ void __launch_bounds__(kThreads, TS == 128 ? 1 : 2)
    fp8_short_kernel(const __grid_constant__ CUtensorMap mapL, const __grid_constant__ CUtensorMap mapS,
                     const __grid_constant__ Fp8ShortParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], done[kMaxStages];
  // accumulators: 4 where two CTAs' fit, no more than stages (a stage's second commit must not precede the
  // folders' look at its first)
  constexpr int kBufs = TS == 128 ? 2 : 4;
  const int bufs = min(kBufs, p.stages);
  __shared__ __align__(8) uint64_t acc_empty[kBufs];
  __shared__ __align__(8) uint64_t scale_full[kChunks], scale_empty[kChunks];
  __shared__ uint32_t tmem_slot;

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  float* share = reinterpret_cast<float*>(smem_raw + pad);  // over the ring, once it is drained
  float* chunks = reinterpret_cast<float*>(smem_raw + pad + p.stages * p.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % p.split;  // of the cluster: blocks of a cluster are consecutive
  const int tile = (int)blockIdx.x / p.split;
  const int l0 = (tile / p.tiles_s) * BL, s0 = (tile % p.tiles_s) * TS;
  const int groups = (p.K + BK - 1) / BK;
  const int g0 = (int)((int64_t)groups * rank / p.split), g1 = (int)((int64_t)groups * (rank + 1) / p.split);
  const int units = g1 - g0;
  constexpr uint32_t kAccCols = TS < 32 ? 32u : (uint32_t)TS;
  constexpr uint32_t kTmemCols = kBufs * kAccCols;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    prefetch_tensormap(&mapL);
    prefetch_tensormap(&mapS);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&done[s]), 1);
    }
    for (int b = 0; b < kBufs; ++b) mbar_init(smem_addr(&acc_empty[b]), kFoldWarps);
    for (int c = 0; c < kChunks; ++c) {
      mbar_init(smem_addr(&scale_full[c]), 32);
      mbar_init(smem_addr(&scale_empty[c]), kFoldWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  // launched as a programmatic dependent: what the stream's kernel before this one wrote is read, and
  // what it read is written, only from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");

  float2 sum[TS / 2];
  const int row = 32 * (warp & 3) + lane;  // of the tile, of a fold thread
  if (warp == 0) {
    // ------------------------------------------------ loads
    const uint32_t bytes = (uint32_t)(BL * BK + (p.s_mn ? 128 * BK : TS * BK));
    int t = 0, s = 0;
    uint32_t lap = 0;
    for (; t < units; ++t) {
      if (lap > 0 && !poll_wait(smem_addr(&done[s]), (lap - 1) & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
        break;
      }
      if (elect_one()) {
        const int k0 = (g0 + t) * BK;
        const uint32_t bar = smem_addr(&full[s]), a = sbase + (uint32_t)(s * p.stage_bytes);
        mbar_arrive_expect_tx(bar, bytes);
        tma_load_3d(a, &mapL, bar, p.l_mn ? l0 : k0, p.l_mn ? k0 : l0, 0);
        tma_load_3d(a + BL * BK, &mapS, bar, p.s_mn ? s0 : k0, p.s_mn ? k0 : s0, 0);
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
    const uint32_t lstep = step_of(p.l_mn), sstep = step_of(p.s_mn), desc0 = desc_lo(sbase);
    int t = 0, s = 0, b = 0;
    uint32_t lap = 0, b_lap = 0;
    for (; t < units; ++t) {
      if ((b_lap > 0 && !poll_wait(smem_addr(&acc_empty[b]), (b_lap - 1) & 1u, p.timeout_ns)) ||
          !poll_wait(smem_addr(&full[s]), lap & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        break;
      }
      tmem_fence_after_sync();
      if (elect_one()) {
        const uint32_t ld = desc0 + (uint32_t)(s * (p.stage_bytes >> 4)), sd = ld + ((BL * BK) >> 4);
#pragma unroll
        for (uint32_t ks = 0; ks < BK / 32; ++ks)
          mma_f8(tmem + (uint32_t)b * kAccCols, make_desc(ld + ks * lstep), make_desc(sd + ks * sstep), p.idesc,
                 ks == 0 ? 0u : 1u);
        mma_commit(smem_addr(&done[s]));  // the stage is free, the accumulator holds group t
      }
      __syncwarp();
      if (++b == bufs) {
        b = 0;
        ++b_lap;
      }
      if (++s == p.stages) {
        s = 0;
        ++lap;
      }
    }
    // leave only when every product has completed and its commit has landed
    bool ok = true;
    for (int u = t > p.stages ? t - p.stages : 0; u < t; ++u)
      ok = ok && poll_wait(smem_addr(&done[u % p.stages]), (uint32_t)(u / p.stages) & 1u, p.timeout_ns);
    if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else if (warp == 2) {
    // ------------------------------------------------ scales of the tile's rows and columns
    const uint32_t ring = smem_addr(chunks);
    int c = 0;
    uint32_t lap = 0;
    for (int t = 0; t < units; t += kChunkGroups) {
      if (lap > 0 && !poll_wait(smem_addr(&scale_empty[c]), (lap - 1) & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
        break;
      }
      const int count = min(kChunkGroups, units - t);
      const uint32_t dst = ring + 4u * (uint32_t)(c * chunk_floats(TS));
      for (int j = lane; j < BL + TS; j += 32) {
        const Fp8Scales& sc = j < BL ? p.sl : p.ss;
        const int64_t at = j < BL ? min(l0 + j, p.L - 1) : min(s0 + j - BL, p.S - 1);
        const int64_t src = (at >> sc.shift) * sc.si + (int64_t)(g0 + t) * sc.sk, n = extent(sc, j < BL ? p.L : p.S, groups);
        for (int g = 0; g < count; ++g)
          copy4_async(p.out.guard, kSiteScale, dst + 4u * (uint32_t)(g * (BL + TS) + j), sc.p, src + (int64_t)g * sc.sk, n);
      }
      copies_arrive(smem_addr(&scale_full[c]));
      if (++c == kChunks) {
        c = 0;
        ++lap;
      }
    }
    copies_wait_all();
  } else if (warp >= kFirstFold) {
    // ------------------------------------------------ folders: a row of the tile each, all its columns
    const uint32_t tq = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll
    for (int e = 0; e < TS / 2; ++e) sum[e] = make_float2(0.0f, 0.0f);
    bool ok = true;
    int s = 0, c = 0, b = 0;
    uint32_t s_lap = 0, c_lap = 0;
    for (int t = 0; t < units; ++t) {
      const int in_chunk = t & (kChunkGroups - 1);
      if (in_chunk == 0) ok = poll_wait(smem_addr(&scale_full[c]), c_lap & 1u, p.timeout_ns);
      ok = ok && poll_wait(smem_addr(&done[s]), s_lap & 1u, p.timeout_ns);
      if (!ok) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        break;
      }
      tmem_fence_after_sync();
      const float* sc = chunks + c * chunk_floats(TS) + in_chunk * (BL + TS);
      const float l = sc[row];
      const float2 l2 = make_float2(l, l);
      constexpr int kCols = TS < 32 ? TS : 32;
#pragma unroll
      for (int j0 = 0; j0 < TS; j0 += kCols) {
        float v[kCols];
        tmem_ld(tq + (uint32_t)b * kAccCols + (uint32_t)j0, v);
        tmem_wait_ld();
        if (j0 + kCols == TS) {
          tmem_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&acc_empty[b]));
        }
#pragma unroll
        for (int j = 0; j < kCols; ++j) asm volatile("" : "+f"(v[j]));  // used behind the wait only
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(sc + BL + j0 + j);
          float2* m = &sum[(j0 + j) / 2];
          // the two scales first: either alone may be far from 1
          m[0] = __ffma2_rn(make_float2(v[j], v[j + 1]), __fmul2_rn(make_float2(w.x, w.y), l2), m[0]);
          m[1] = __ffma2_rn(make_float2(v[j + 2], v[j + 3]), __fmul2_rn(make_float2(w.z, w.w), l2), m[1]);
        }
      }
      if (in_chunk == kChunkGroups - 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&scale_empty[c]));
        if (++c == kChunks) {
          c = 0;
          ++c_lap;
        }
      }
      if (++b == bufs) b = 0;
      if (++s == p.stages) {
        s = 0;
        ++s_lap;
      }
    }
  }

  // ------------------------------------------------ the shares, added in rank order
  tmem_fence_before_sync();
  __syncthreads();  // the ring is drained: loads have landed and the products that read it are done
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (warp >= kFirstFold) {
    const int sl = p.trans ? 1 : share_pitch(false, TS), ss = p.trans ? share_pitch(true, TS) : 1;
#pragma unroll
    for (int e = 0; e < TS / 2; ++e) {
      share[2 * e * ss + row * sl] = sum[e].x;
      share[(2 * e + 1) * ss + row * sl] = sum[e].y;
    }
  }
  __syncthreads();
  if (p.split > 1) cluster_sync();
  // this CTA's part of the tile: its share of the columns (D transposed: lanes along the long side)
  // or of the rows (lanes along the short side, the columns of D)
  const int nl = min(BL, p.L - l0), ns = min(TS, p.S - s0);
  const int parts = p.trans ? ns : nl;
  const int b0 = parts * rank / p.split, b1 = parts * (rank + 1) / p.split;
  const int inner = p.trans ? BL : TS;  // powers of two
  const int shift = 31 - __clz(inner);
  for (int i = (int)threadIdx.x; i < (b1 - b0) << shift; i += kThreads) {
    const int outer_i = b0 + (i >> shift), inner_i = i & (inner - 1);
    const int l = p.trans ? inner_i : outer_i, s = p.trans ? outer_i : inner_i;
    if (l >= nl || s >= ns) continue;
    const int word = outer_i * share_pitch(p.trans, TS) + inner_i;
    const uint32_t at = sbase + 4u * (uint32_t)word;
    float v = 0.0f;
    if (p.split == 1) {
      v = share[word];
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

// f(kernel) for a tile width.
template <typename F>
cudaError_t with_short_kernel(int tile_s, const F& f) {
  switch (tile_s) {
    case 16: return f(fp8_short_kernel<16>);
    case 32: return f(fp8_short_kernel<32>);
    case 64: return f(fp8_short_kernel<64>);
    case 128: return f(fp8_short_kernel<128>);
  }
  return cudaErrorInvalidValue;
}

__global__ void __launch_bounds__(256) repack_kernel(const uint8_t* __restrict__ src, int64_t ld, int64_t rows,
                                                     int64_t cols, uint8_t* __restrict__ dst, int64_t ldd,
                                                     const Guard guard) {
  const int64_t chunks = ldd / 16, total = rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / chunks, c = (i - r * chunks) * 16;
    const int64_t s = r * ld + c;
    const int n = (int)min((int64_t)16, cols - c);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k < n) w[k / 4] |= (uint32_t)get_at(guard, kSiteCodes, src, s + k, extent(rows, ld, cols)) << (8 * (k % 4));
    put_at(guard, kSitePart, reinterpret_cast<uint4*>(dst), i, total, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

__global__ void __launch_bounds__(256) scale_kernel(const Fp8Out o) {
  const int64_t total = (int64_t)o.M * o.N;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / o.N, col = i - row * o.N;
    const float x = o.beta == 0.0f ? 0.0f : o.beta * read_c(o, row, col);
    if (!d_holds(o, row, col, 1)) continue;
    const int64_t d = row * o.ldd + col;
    if (o.bf16) static_cast<__nv_bfloat16*>(o.D)[d] = __float2bfloat16_rn(x);
    else        static_cast<float*>(o.D)[d] = x;
  }
}

}  // namespace
}  // namespace f8

size_t fp8_short_smem(int tile_s, int stages, int stage_bytes) {
  const size_t ring = (size_t)stages * stage_bytes + (size_t)f8::kChunks * f8::chunk_floats(tile_s) * 4;
  const size_t share = (size_t)f8::share_words(tile_s) * 4;
  return (ring > share ? ring : share) + 1024;
}

cudaError_t prepare_fp8_short() {
  for (int tile_s : kFp8ShortTiles) {
    const cudaError_t e = f8::with_short_kernel(tile_s, [](auto kernel) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, f8::kMaxSmem);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_fp8_short(const CUtensorMap& mapL, const CUtensorMap& mapS, const Fp8ShortParams& p,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tiles_l * p.tiles_s * p.split));
  cfg.blockDim = dim3(f8::kThreads);
  cfg.dynamicSmemBytes = fp8_short_smem(p.tile_s, p.stages, p.stage_bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return f8::with_short_kernel(p.tile_s,
                               [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, mapL, mapS, p); });
}

cudaError_t launch_fp8_repack(const void* src, int64_t ld, int64_t rows, int64_t cols, void* dst, int64_t ldd,
                              const Guard& guard, cudaStream_t stream) {
  const int64_t blocks = (rows * (ldd / 16) + 255) / 256;
  f8::repack_kernel<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(
      static_cast<const uint8_t*>(src), ld, rows, cols, static_cast<uint8_t*>(dst), ldd, guard);
  return cudaGetLastError();
}

cudaError_t launch_fp8_scale(const Fp8Out& o, cudaStream_t stream) {
  const int64_t blocks = ((int64_t)o.M * o.N + 255) / 256;
  f8::scale_kernel<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(o);
  return cudaGetLastError();
}

}  // namespace sgemm_impl
