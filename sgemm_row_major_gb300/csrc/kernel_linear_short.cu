// kernel_linear_short.cu -- products of BF16 matrices with few rows, for sm_103a, with what a layer does to the sums.
//
// The products of kernel_linear_pair.cu where the time is that of reading the weights (a decoding step).  The columns of D run
// along the 128 rows of the tensor core and its few rows (tokens) along the columns (TS 16, 32, 64 or 128), so one token costs
// a 128 x 16 tile and not a 256-row one; gated, a CTA holds 128 rows of gate and the same 128 of up.  A cluster of `split`
// CTAs (1, 2, 4 or 8) divides the K of a tile; each leaves its sums in shared memory and the cluster adds the shares in rank
// order, each CTA the tokens of its part, read from its peers' shared memory: no workspace, one launch, and the same result
// every time.  A warp writes 128 columns of one token at a time, which are one group of what is kept in 8 bits.
//
// Warp 0 loads (TMA), warp 1 issues the products, warps 4-7 take the accumulators to FP32 registers, all warps join the shares.  Two CTAs
// share an SM where their sums leave room.
//
// Bound by reading the weights and, below about 20 us, by the start, the first loads and the joining: 64 x 16384 -> 4096 takes
// 27.6 us, 4.9 TB/s; gated 1 x 4096 -> 8192 25.7 us, 5.2 TB/s; 1 x 4096 -> 4096 10.3 us, 3.3 TB/s.
#include "linear_common.cuh"

namespace sgemm_impl {
namespace lin {
namespace {

using namespace tc;

constexpr int BL = 128, BK = 64;
constexpr int kFirstFold = 4, kFoldWarps = 4;
constexpr int kThreads = 32 * (kFirstFold + kFoldWarps);
constexpr int kMaxStages = kLinearShortMaxStages;
static_assert(kThreads == kLinearShortThreads, "the plan's figure");
constexpr int kMaxSmem = 220 * 1024;
constexpr int kFold = 8;  // K tiles that are summed in one accumulator (their sums drift: kernel_linear_pair.cu)
constexpr int kPitch = BL + 4;  // words from token to token of a share: reads and writes of 32 lanes hit different banks
__host__ __device__ constexpr int share_bytes(int tile_s, bool gated) { return (gated ? 2 : 1) * tile_s * kPitch * 4; }

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// What is kept of 4 columns of a token; all lanes of the warp, which hold 128 columns (n < 1: none here).
__device__ __forceinline__ void keep4(const LinearOut& o, const LinearJob& j, int which, int row, int col, int n, const float (&v)[4]) {
  const LinearKept& k = o.kept[which];
  if (o.keep == 1) {
    if (n > 0 && kept_ok(o, j, which, row, col, n)) put4(static_cast<__nv_bfloat16*>(k.data) + (int64_t)row * k.ld + col, n, o.kept_vec8[which], v);
    return;
  }
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) m = fmaxf(m, e < n ? f8::finite_abs(v[e]) : 0.0f);
  const float scale = f8::group_scale(f8::lanes_max<32>(m), kMaxE4M3), inv = __fdiv_rn(1.0f, scale);
  if (n <= 0) return;
  if (col % 128 == 0) put_scale(o, j, which, row, col >> 7, scale);
  const uint32_t u = f8::codes2<true>(v[0] * inv, v[1] * inv, false) | (f8::codes2<true>(v[2] * inv, v[3] * inv, false) << 16);
  if (!kept_ok(o, j, which, row, col, n)) return;
  uint8_t* d = static_cast<uint8_t*>(k.data) + (int64_t)row * k.ld + col;
  if (k.vec && n == 4) {
    *reinterpret_cast<uint32_t*>(d) = u;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) d[e] = (uint8_t)(u >> (8 * e));
  }
}

template <int TS, bool GATED>
__global__ void __launch_bounds__(kThreads, GATED || TS == 128 ? 1 : 2)
    linear_short_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearShortParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kParts = GATED ? 2 : 1;
  constexpr uint32_t kAccCols = TS < 32 ? 32u : (uint32_t)TS;
  constexpr int kBufs = 2;
  constexpr uint32_t kTmemCols = kBufs * kParts * kAccCols;
  __shared__ __align__(8) uint64_t full[kMaxStages], done[kMaxStages];
  __shared__ __align__(8) uint64_t acc_full[kBufs], acc_empty[kBufs];
  __shared__ uint32_t tmem_slot;

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  float* share = reinterpret_cast<float*>(smem_raw + pad);  // over the ring, once it is drained
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % p.split;  // of the cluster: blocks of a cluster are consecutive
  const int tile = (int)blockIdx.x / p.split;
  const LinearJob& j = p.job;
  const int l0 = (tile / j.tiles_m) * BL, s0 = (tile % j.tiles_m) * TS;
  const int kt = j.k_tiles * j.segments;
  const int g0 = (int)((int64_t)kt * rank / p.split), g1 = (int)((int64_t)kt * (rank + 1) / p.split);
  const int units = g1 - g0;

  if (threadIdx.x == 0) {
    prefetch_tensormap(&maps.op[j.a[0]]);
    prefetch_tensormap(&maps.op[j.b[0]]);
    if (GATED) prefetch_tensormap(&maps.op[j.b[1]]);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&done[s]), 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(smem_addr(&acc_full[b]), 1);
      mbar_init(smem_addr(&acc_empty[b]), kFoldWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  // Not before this CTA has its tensor memory: a dependent that took it first would wait for this grid, and this grid for it.
  // (As a dependent itself it takes at most 256 columns: no kernel of the library that needs more than the others leaves its
  // shared memory.)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // launched as a programmatic dependent: what the stream's kernel before this one wrote is read, and what it read is
  // written, only from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");

  float sum[kParts * TS];
  if (warp == 0) {
    // ------------------------------------------------ loads
    int t = 0, s = 0;
    uint32_t lap = 0;
    for (; t < units; ++t) {
      if (lap > 0 && !poll_wait(smem_addr(&done[s]), (lap - 1) & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
        break;
      }
      if (elect_one()) {
        const int segment = g0 + t >= j.k_tiles, k0 = (g0 + t - segment * j.k_tiles) * BK;
        const uint32_t bar = smem_addr(&full[s]), l = sbase + (uint32_t)(s * p.stage_bytes);
        const auto load = [&](uint32_t dst, const CUtensorMap* map, int inner, int outer) { tma_load_3d(dst, map, bar, inner, outer, 0); };
        mbar_arrive_expect_tx(bar, (uint32_t)p.stage_bytes);
        load_part(load, l, &maps.op[j.b[GATED ? 0 : segment]], j.b_mn, l0, k0, BL);
        if (GATED) load_part(load, l + BL * BK * 2, &maps.op[j.b[1]], j.b_mn, l0, k0, BL);
        load_part(load, l + kParts * BL * BK * 2, &maps.op[j.a[segment]], j.a_mn, s0, k0, TS);
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
    const uint32_t lstep = step_of(j.b_mn), sstep = step_of(j.a_mn), desc0 = desc_lo(sbase);
    int t = 0, s = 0, b = 0;
    uint32_t lap = 0, b_lap = 0;
    bool ok = true;
    while (ok && t < units) {
      const int n = min(kFold, units - t);
      ok = b_lap == 0 || poll_wait(smem_addr(&acc_empty[b]), (b_lap - 1) & 1u, p.timeout_ns);
      tmem_fence_after_sync();
      for (int i = 0; ok && i < n; ++i) {
        ok = poll_wait(smem_addr(&full[s]), lap & 1u, p.timeout_ns);
        if (!ok) break;
        tmem_fence_after_sync();
        if (elect_one()) {
          const uint32_t ld = desc0 + (uint32_t)(s * (p.stage_bytes >> 4));
          const uint32_t sd = ld + (uint32_t)(kParts * BL * BK * 2 >> 4);
#pragma unroll
          for (int w = 0; w < kParts; ++w)
#pragma unroll
            for (uint32_t ks = 0; ks < BK / 16; ++ks)
              mma_bf16(tmem + (uint32_t)(b * kParts + w) * kAccCols, make_desc(ld + (uint32_t)(w * (BL * BK * 2 >> 4)) + ks * lstep),
                       make_desc(sd + ks * sstep), j.idesc, i == 0 && ks == 0 ? 0u : 1u);
          f8::mma_commit(smem_addr(&done[s]));
          if (i == n - 1) f8::mma_commit(smem_addr(&acc_full[b]));
        }
        __syncwarp();
        ++t;
        if (++s == p.stages) {
          s = 0;
          ++lap;
        }
      }
      if (++b == kBufs) {
        b = 0;
        ++b_lap;
      }
    }
    if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
    // leave only when every product has completed and its commit has landed
    ok = true;
    for (int u = t > p.stages ? t - p.stages : 0; u < t; ++u)
      ok = ok && poll_wait(smem_addr(&done[u % p.stages]), (uint32_t)(u / p.stages) & 1u, p.timeout_ns);
    if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else if (warp >= kFirstFold) {
    // ------------------------------------------------ folders: a column of D each, all its tokens
    const uint32_t tq = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll
    for (int e = 0; e < kParts * TS; ++e) sum[e] = 0.0f;
    int b = 0;
    uint32_t b_lap = 0;
    for (int t = 0; t < units; t += kFold) {
      if (!poll_wait(smem_addr(&acc_full[b]), b_lap & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        break;
      }
      tmem_fence_after_sync();
      constexpr int kCols = TS < 32 ? TS : 32;
#pragma unroll
      for (int w = 0; w < kParts; ++w)
#pragma unroll
        for (int j0 = 0; j0 < TS; j0 += kCols) {
          float v[kCols];
          f8::tmem_ld(tq + (uint32_t)(b * kParts + w) * kAccCols + (uint32_t)j0, v);
          tmem_wait_ld();
          if (w == kParts - 1 && j0 + kCols == TS) {
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&acc_empty[b]));
          }
          tmem_ld_ready(v);
#pragma unroll
          for (int k = 0; k < kCols; ++k) sum[w * TS + j0 + k] += v[k];
        }
      if (++b == kBufs) {
        b = 0;
        ++b_lap;
      }
    }
  }

  // ------------------------------------------------ the shares, added in rank order
  tmem_fence_before_sync();
  __syncthreads();  // the ring is drained: loads have landed and the products that read it are done
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (warp >= kFirstFold) {
    const int l = 32 * (warp & 3) + lane;
#pragma unroll
    for (int e = 0; e < kParts * TS; ++e) share[e * kPitch + l] = sum[e];
  }
  __syncthreads();
  if (p.split > 1) cluster_sync();
  // this CTA's tokens of the tile: a warp per token, 4 columns per lane
  const LinearOut& o = p.out;
  const int ns = min(TS, j.M - s0);
  const int b0 = ns * rank / p.split, b1 = ns * (rank + 1) / p.split;
  const int col = l0 + 4 * lane, n = min(4, j.N - col);
  for (int s = b0 + warp; s < b1; s += kThreads / 32) {
    float v[kParts][4];
#pragma unroll
    for (int w = 0; w < kParts; ++w) {
      const uint32_t at = sbase + 4u * (uint32_t)((w * TS + s) * kPitch + 4 * lane);
      float4 u[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < p.split) u[r] = ld_cluster4(p.split > 1 ? map_to_rank(at, (uint32_t)r) : at);
      float4 x = u[0];
#pragma unroll
      for (int r = 1; r < 8; ++r)
        if (r < p.split) x = make_float4(x.x + u[r].x, x.y + u[r].y, x.z + u[r].z, x.w + u[r].w);
      v[w][0] = x.x;
      v[w][1] = x.y;
      v[w][2] = x.z;
      v[w][3] = x.w;
    }
    const int row = s0 + s;
    if (!GATED && o.bias && n > 0 && in_range(o.guard.fault, o.guard.word, f8::kSiteIn, col, n, j.N)) {
      float x[4];
      get4(static_cast<const __nv_bfloat16*>(o.bias) + col, n, o.bias_vec, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][e] += x[e];
    }
    if (o.keep) {
      keep4(o, j, 0, row, col, n, v[0]);
      if constexpr (GATED) keep4(o, j, 1, row, col, n, v[kParts - 1]);
    }
    if (n <= 0) continue;
    with_act(o.act, [&](auto act) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float2 f = act_of<decltype(act)::value>(make_float2(v[0][e], v[0][e + 1]));
        if (GATED) f = mul(f, make_float2(v[kParts - 1][e], v[kParts - 1][e + 1]));
        v[0][e] = f.x;
        v[0][e + 1] = f.y;
      }
    });
    if (!GATED && o.residual && r_ok(o, j, row, col, n)) {
      float x[4];
      get4(static_cast<const __nv_bfloat16*>(o.residual) + (int64_t)row * o.ldr + col, n, o.r_vec, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][e] += x[e];
    }
    put_row(o, j, row, col, n, v[0]);
  }
  if (p.split > 1) {
    __syncthreads();
    cluster_sync();  // no CTA leaves while a peer may read its share
  }
}

// f(kernel) for a tile width and form.
template <typename F>
cudaError_t with_kernel(int tile_s, bool gated, const F& f) {
  switch (tile_s) {
    case 16: return gated ? f(linear_short_kernel<16, true>) : f(linear_short_kernel<16, false>);
    case 32: return gated ? f(linear_short_kernel<32, true>) : f(linear_short_kernel<32, false>);
    case 64: return gated ? f(linear_short_kernel<64, true>) : f(linear_short_kernel<64, false>);
    case 128: return gated ? cudaErrorInvalidValue : f(linear_short_kernel<128, false>);
  }
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace lin

int64_t linear_short_smem(int tile_s, bool gated, int stages, int stage_bytes) {
  const int64_t ring = (int64_t)stages * stage_bytes, share = lin::share_bytes(tile_s, gated);
  return (ring > share ? ring : share) + 1024;
}

cudaError_t prepare_linear_short() {
  for (int tile_s : kLinearShortTiles)
    for (int gated = 0; gated < 2; ++gated) {
      if (gated && tile_s == 128) continue;
      const cudaError_t e = lin::with_kernel(tile_s, gated != 0, [](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, lin::kMaxSmem);
      });
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

cudaError_t launch_linear_short(bool gated, const LinearMaps& maps, const LinearShortParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.job.tiles_n * p.job.tiles_m * p.split));
  cfg.blockDim = dim3(lin::kThreads);
  cfg.dynamicSmemBytes = (size_t)linear_short_smem(p.tile_s, gated, p.stages, p.stage_bytes);
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
  return lin::with_kernel(p.tile_s, gated, [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, maps, p); });
}

}  // namespace sgemm_impl
