// kernel_fp8_moe.cu -- a mixture-of-experts layer for a few tokens on 8-bit weights, for sm_103a.
//
//     Y_t = sum_{e chosen by t} c_te W2_e (silu(W1_e x_t) * (W3_e x_t))
//
// Two kernels, both streams of the chosen experts' weights: every weight tile is loaded once and
// meets all the tokens that need it, as the 128 rows of a tensor-core product whose columns are
// tokens (16 to 64 of them, so the products cost little beside the loads).
//
// moe_up_kernel: every CTA works out the routing from the logits by itself (a warp per token; top_k
// rounds of a warp maximum), which costs less than a launch, and takes tiles of 64 inner columns of
// active experts: rows 0-63 of the product are rows of W1_e, rows 64-127 rows of W3_e, the columns
// all the tokens in order, so x is loaded as it lies and no token is gathered.  The sums of the
// tokens that chose e become h = silu(gate) * up, stored as two E4M3 terms with a scale per 64
// columns: hi = rn8(h / s), lo = rn8(16 (h / s - hi)), together within 2^-9.8 of the group's largest
// value.  As the second product is bound by the weights, the doubled columns are free.
//
// moe_down_kernel: a cluster of CTAs per 128 rows of the hidden side shares the (expert, 128 inner
// columns) units in order; each CTA folds its units per expert in FP32 registers, adds them weighted
// into its tokens' sums in shared memory, and the cluster adds those in rank order into Y.
//
// Both: warp 0 loads (TMA), warp 1 issues the products, warps 2-5 fold; two CTAs per SM.
#include <algorithm>

#include "fp8_gemm.cuh"

namespace sgemm_impl {
namespace f8 {
namespace {

using namespace tc;

constexpr int BK = 128;
constexpr int kThreads = 192, kFoldThreads = 128;
constexpr int kMaxStages = 8;
constexpr int kWTile = 128 * BK;  // 16 KB of weights per stage
constexpr int kUpCols = 64;       // inner columns of a tile of the first kernel
constexpr float kLoScale = 16.0f;
constexpr int kPitch = 129;

__device__ __forceinline__ void fold_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ uint32_t moe_idesc(int n) {  // E4M3, K-major, FP32 accumulator, M = 128
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// Total order of floats as unsigned integers; NaN is mapped to 0 (below -Inf) by the caller.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Routing arrays in shared memory.
struct Route {
  int n;                       // active experts
  unsigned long long* mask;    // [active]
  int *expert, *base;          // [active]
};

// Bytes of dynamic shared memory the first kernel's routing takes.
__host__ __device__ inline size_t up_route_bytes(const MoeParams& p) {
  return (size_t)p.experts * 8 + (size_t)p.active_max * 16 + (size_t)p.tokens * p.top_k * 8;
}
__host__ __device__ inline size_t down_route_bytes(const MoeParams& p) {
  return (size_t)p.active_max * 8 + (size_t)p.slots_max * 8;
}
__host__ __device__ inline int token_cols(const MoeParams& p) { return (p.tokens + 15) / 16 * 16; }
__host__ __device__ inline size_t up_stage_bytes(const MoeParams& p) { return kWTile + (size_t)token_cols(p) * BK; }
__host__ __device__ inline size_t down_stage_bytes(const MoeParams& p) {
  return kWTile + (size_t)2 * token_cols(p) * BK;
}
__host__ __device__ inline size_t up_smem(const MoeParams& p) {
  return 1024 + p.up_stages * up_stage_bytes(p) + (size_t)p.tokens * kPitch * 4 + 16 + up_route_bytes(p);
}
__host__ __device__ inline size_t down_smem(const MoeParams& p) {
  return 1024 + p.down_stages * down_stage_bytes(p) + (size_t)p.tokens * 128 * 4 + down_route_bytes(p);
}

// top_k experts of token t by one warp: experts and softmax weights to chosen / weight (expert -1
// where there is none), 1 to *poisoned for a NaN or +Inf logit.
__device__ void route_token(const MoeParams& p, int t, int* chosen, float* weight, int* poisoned) {
  constexpr int kPer = kMoeMaxExperts / 32;
  const int lane = threadIdx.x & 31;
  const float* row = p.logits + (int64_t)t * p.ldl;
  const int per = (p.experts + 31) / 32;
  uint32_t key[kPer];  // expert e = 32 i + lane
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    key[i] = 0u;
    if (i < per && 32 * i + lane < p.experts) {
      const float x = row[32 * i + lane];
      if (!(x < INFINITY)) bad = true;
      else if (x > -INFINITY) key[i] = order_key(x + 0.0f);  // -0 counts as 0
    }
  }
  if (lane == 0) *poisoned = 0;
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) *poisoned = 1;
    for (int j = lane; j < p.top_k; j += 32) chosen[j] = -1;
    return;
  }
  float top = 0.0f, sum = 0.0f;
  float mine = 0.0f;  // lane j: exp(logit - top) of choice j
  int mine_e = -1;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per && key[i] > best) {  // the first of equals: the lowest index of this lane
        best = key[i];
        at = i;
      }
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    if (most == 0u) break;  // no expert with a finite logit is left
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == most ? (uint32_t)(32 * at + lane) : 0xffffffffu);
    const uint32_t bits = most & 0x80000000u ? most & 0x7FFFFFFFu : ~most;
    const float x = __uint_as_float(bits);
    if (j == 0) {
      top = x;
      if (!p.renormalize) {  // over all experts
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i < per && key[i] != 0u) {
            const uint32_t k = key[i];
            s += expf(__uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k) - top);
          }
        sum = warp_sum(s);
      }
    }
    const float w = expf(x - top);
    if (p.renormalize) sum += w;
    if (lane == j) {
      mine = w;
      mine_e = (int)e;
    }
    if ((int)(e & 31u) == lane) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == (int)(e >> 5)) key[i] = 0u;
    }
  }
  if (lane < p.top_k) {
    chosen[lane] = mine_e;
    weight[lane] = mine / sum;
  }
}

__global__ void __launch_bounds__(kThreads, 2) moe_up_kernel(const __grid_constant__ CUtensorMap mapX,
                                                             const __grid_constant__ CUtensorMap mapG,
                                                             const __grid_constant__ CUtensorMap mapU,
                                                             const __grid_constant__ MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int n_active;
  __shared__ int poisoned[kMoeMaxTokens];
  __shared__ __align__(16) float col_scale[2][kFoldThreads];

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  const int stage_bytes = (int)up_stage_bytes(p);
  const int ncols = token_cols(p);
  float* sums = reinterpret_cast<float*>(smem_raw + pad + p.up_stages * stage_bytes);  // [slot of the expert][kPitch]
  unsigned long long* mask_of =  // [experts], then the active experts' arrays
      reinterpret_cast<unsigned long long*>((reinterpret_cast<uintptr_t>(sums + p.tokens * kPitch) + 15) & ~uintptr_t(15));
  Route r;
  r.mask = mask_of + p.experts;
  r.expert = reinterpret_cast<int*>(r.mask + p.active_max);
  r.base = r.expert + p.active_max;
  int* chosen = r.base + p.active_max;  // [tokens][top_k]
  float* weight = reinterpret_cast<float*>(chosen + p.tokens * p.top_k);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.up_stages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&acc_full[b]), 1);
      mbar_init(smem_addr(&acc_empty[b]), kFoldThreads / 32);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), 128);
  // ------------------------------------------------ routing
  for (int e = (int)threadIdx.x; e < p.experts; e += kThreads) mask_of[e] = 0ull;
  for (int t = warp; t < p.tokens; t += kThreads / 32)
    route_token(p, t, chosen + t * p.top_k, weight + t * p.top_k, &poisoned[t]);
  __syncthreads();
  for (int i = (int)threadIdx.x; i < p.tokens * p.top_k; i += kThreads)
    if (chosen[i] >= 0) {
      const int t = i / p.top_k;
      atomicOr(reinterpret_cast<unsigned*>(&mask_of[chosen[i]]) + (t >> 5), 1u << (t & 31));
    }
  __syncthreads();
  if (warp == 0) {  // active experts in ascending order, 32 at a time
    int n = 0, slots = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + lane;
      const unsigned long long m = e < p.experts ? mask_of[e] : 0ull;
      const unsigned act = __ballot_sync(0xffffffffu, m != 0ull);
      int c = __popcll(m), before = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
      }
      if (m != 0ull) {
        const int a = n + __popc(act & ((1u << lane) - 1u));
        r.mask[a] = m;
        r.expert[a] = e;
        r.base[a] = slots + before - c;
      }
      n += __popc(act);
      slots += __shfl_sync(0xffffffffu, before, 31);
    }
    if (lane == 0) n_active = n;
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  r.n = n_active;
  if (blockIdx.x == 0) {  // the second kernel's copy
    if (threadIdx.x == 0) p.route.counts[0] = r.n;
    for (int a = (int)threadIdx.x; a < r.n; a += kThreads) {
      p.route.expert[a] = r.expert[a];
      p.route.base[a] = r.base[a];
      p.route.mask[a] = r.mask[a];
      unsigned long long m = r.mask[a];
      for (int j = 0; m != 0ull; ++j, m &= m - 1ull) {
        const int t = __ffsll((long long)m) - 1;
        float w = 0.0f;
        for (int i = 0; i < p.top_k; ++i)
          if (chosen[t * p.top_k + i] == r.expert[a]) w = weight[t * p.top_k + i];
        p.route.slot_token[r.base[a] + j] = t;
        p.route.slot_weight[r.base[a] + j] = w;
      }
    }
    for (int t = (int)threadIdx.x; t < p.tokens; t += kThreads) p.route.poisoned[t] = poisoned[t];
  }

  const int col_tiles = (p.inner + kUpCols - 1) / kUpCols;
  const int items = r.n * col_tiles;
  const int my_items = (int)blockIdx.x < items ? (items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
  const int groups = (p.hidden + BK - 1) / BK;

  if (warp == 0) {
    const uint32_t bytes = (uint32_t)stage_bytes;
    int t = 0, s = 0;
    uint32_t lap = 0;
    bool ok = true;
    for (int i = 0; ok && i < my_items; ++i) {
      const int item = (int)blockIdx.x + i * (int)gridDim.x;
      const int e = r.expert[item / col_tiles], c0 = (item % col_tiles) * kUpCols;
      for (int g = 0; g < groups; ++g, ++t) {
        if (lap > 0 && !poll_wait(smem_addr(&empty[s]), (lap - 1) & 1u, p.timeout_ns)) {
          if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t bar = smem_addr(&full[s]), a = sbase + (uint32_t)(s * stage_bytes);
          mbar_arrive_expect_tx(bar, bytes);
          tma_load_3d(a, &mapG, bar, g * BK, c0, e);
          tma_load_3d(a + kWTile / 2, &mapU, bar, g * BK, c0, e);
          tma_load_3d(a + kWTile, &mapX, bar, g * BK, 0, 0);
        }
        if (++s == p.up_stages) {
          s = 0;
          ++lap;
        }
      }
    }
    for (int u = t > p.up_stages ? t - p.up_stages : 0; u < t; ++u)  // every copy has landed before the CTA ends
      if (!poll_wait(smem_addr(&full[u % p.up_stages]), (uint32_t)(u / p.up_stages) & 1u, p.timeout_ns) && lane == 0)
        atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else if (warp == 1) {
    const uint32_t idesc = moe_idesc(ncols);
    const int units = my_items * groups;
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
        const uint32_t a = sbase + (uint32_t)(s * stage_bytes);
        const uint32_t wd = desc_lo(a), xd = desc_lo(a + kWTile);
#pragma unroll
        for (int ks = 0; ks < BK / 32; ++ks)
          mma_f8(tmem + (uint32_t)b * 64u, make_desc(wd + (uint32_t)ks * step_of(0)),
                 make_desc(xd + (uint32_t)ks * step_of(0)), idesc,
                 ks == 0 ? 0u : 1u);
        mma_commit(smem_addr(&empty[s]));
        mma_commit(smem_addr(&acc_full[b]));
      }
      __syncwarp();
      if (++s == p.up_stages) {
        s = 0;
        ++lap;
      }
    }
    bool ok = true;  // every product has completed, and its commits have landed, before the CTA ends
    for (int u = t > p.up_stages ? t - p.up_stages : 0; u < t; ++u)
      ok = ok && poll_wait(smem_addr(&empty[u % p.up_stages]), (uint32_t)(u / p.up_stages) & 1u, p.timeout_ns);
    for (int u = t > 2 ? t - 2 : 0; u < t; ++u)
      ok = ok && poll_wait(smem_addr(&acc_full[u & 1]), (uint32_t)(u / 2) & 1u, p.timeout_ns);
    if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else {
    const int q = warp & 3;
    const int row = 32 * q + lane;  // rows 0-63: gate, 64-127: up
    const int fid = (int)threadIdx.x - 64;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
    const float* sx = p.sx + (int64_t)min(fid, p.tokens - 1) * p.ldsx;
    bool ok = true;
    int t = 0;
    for (int i = 0; i < my_items; ++i) {
      const int item = (int)blockIdx.x + i * (int)gridDim.x;
      const int a = item / col_tiles, c0 = (item % col_tiles) * kUpCols;
      const int e = r.expert[a];
      const float* sw = row < 64 ? p.sg + (int64_t)e * p.stride_sg + (int64_t)(c0 >> 7) * p.ldsg
                                 : p.su + (int64_t)e * p.stride_su + (int64_t)(c0 >> 7) * p.ldsu;
      float sum[kMoeMaxTokens];
#pragma unroll
      for (int j = 0; j < kMoeMaxTokens; ++j) sum[j] = 0.0f;
      float w_next = __ldg(sw), x_next = __ldg(sx);
      for (int g = 0; g < groups; ++g, ++t) {
        const int b = t & 1;
        const float w_cur = w_next;
        col_scale[b][fid] = x_next;  // last read two groups ago: one barrier per group suffices
        if (g + 1 < groups) {
          w_next = __ldg(sw + g + 1);
          x_next = __ldg(sx + g + 1);
        }
        fold_barrier();
        if (ok) {  // a warp that gave up keeps meeting the others at the barriers
          ok = poll_wait(smem_addr(&acc_full[b]), (uint32_t)(t / 2) & 1u, p.timeout_ns);
          if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        }
        if (!ok) continue;
        tmem_fence_after_sync();
#pragma unroll
        for (int c = 0; c < kMoeMaxTokens / 16; ++c)
          if (16 * c < ncols) {
            float v[16];
            tmem_ld16(tq + (uint32_t)(64 * b + 16 * c), v);
            tmem_wait_ld();
            if (16 * (c + 1) >= ncols) {
              tmem_fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&acc_empty[b]));
            }
            tmem_ld_ready(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[16 * c + j] = fmaf(v[j] * col_scale[b][16 * c + j], w_cur, sum[16 * c + j]);
          }
      }
      // the chosen tokens' sums, compacted, to shared memory; then a warp per slot
      const unsigned long long mask = r.mask[a];
      fold_barrier();  // the previous item's sums have been read
#pragma unroll
      for (int j = 0; j < kMoeMaxTokens; ++j)
        if ((mask >> j) & 1ull) sums[__popcll(mask & ((1ull << j) - 1ull)) * kPitch + row] = sum[j];
      fold_barrier();
      if (!ok) continue;
      const int n = __popcll(mask);
      for (int j = warp - 2; j < n; j += kFoldThreads / 32) {
        const float* s = sums + j * kPitch;
        float h[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float gate = s[2 * lane + k], up = s[64 + 2 * lane + k];
          h[k] = gate / (1.0f + expf(-gate)) * up;
        }
        const float scale = group_scale(lanes_max<32>(fmaxf(finite_abs(h[0]), finite_abs(h[1]))), kMaxE4M3);
        const float inv = __frcp_rn(scale);
        const float v0 = h[0] * inv, v1 = h[1] * inv;
        const uint32_t hi = codes2<true>(v0, v1, false);
        const __half2 back = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3));
        const float2 f = __half22float2(back);
        const uint32_t lo = codes2<true>((v0 - f.x) * kLoScale, (v1 - f.y) * kLoScale, false);
        const int col = c0 + 2 * lane;
        const int64_t slot = r.base[a] + j;
        if (col < p.inner) {  // inner is even
          *reinterpret_cast<uint16_t*>(p.h + 2 * slot * p.inner + col) = (uint16_t)hi;
          *reinterpret_cast<uint16_t*>(p.h + (2 * slot + 1) * p.inner + col) = (uint16_t)lo;
        }
        if (lane == 0) p.sh[slot * p.h_groups + c0 / kUpCols] = scale;
      }
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, 128);
}

__global__ void __launch_bounds__(kThreads, 2) moe_down_kernel(const __grid_constant__ CUtensorMap mapH,
                                                               const __grid_constant__ CUtensorMap mapD,
                                                               const __grid_constant__ MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float col_scale[2][kMoeMaxTokens];

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  const int stage_bytes = (int)down_stage_bytes(p);
  float* ysum = reinterpret_cast<float*>(smem_raw + pad + p.down_stages * stage_bytes);  // [tokens][128]
  int* expert = reinterpret_cast<int*>(ysum + p.tokens * 128);
  int* base = expert + p.active_max;
  int* slot_token = base + p.active_max;
  float* slot_weight = reinterpret_cast<float*>(slot_token + p.slots_max);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % p.split, tile = (int)blockIdx.x / p.split;
  const int l0 = tile * 128;
  const int groups = (p.inner + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.down_stages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&acc_full[b]), 1);
      mbar_init(smem_addr(&acc_empty[b]), kFoldThreads / 32);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), 256);
  for (int i = (int)threadIdx.x; i < p.tokens * 128; i += kThreads) ysum[i] = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel's routing and inner values are complete
  const int n_active = p.route.counts[0];
  for (int a = (int)threadIdx.x; a < n_active; a += kThreads) {
    expert[a] = p.route.expert[a];
    base[a] = p.route.base[a];
  }
  const int n_slots =
      n_active > 0 ? p.route.base[n_active - 1] + __popcll(p.route.mask[n_active - 1]) : 0;
  for (int i = (int)threadIdx.x; i < n_slots; i += kThreads) {
    slot_token[i] = p.route.slot_token[i];
    slot_weight[i] = p.route.slot_weight[i];
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const int total = n_active * groups;
  const int u0 = (int)((int64_t)total * rank / p.split), u1 = (int)((int64_t)total * (rank + 1) / p.split);
  const auto slots_of = [&](int a) { return (a + 1 < n_active ? base[a + 1] : n_slots) - base[a]; };

  if (warp == 0) {
    int t = 0, s = 0;
    uint32_t lap = 0;
    for (int u = u0; u < u1; ++u, ++t) {
      if (lap > 0 && !poll_wait(smem_addr(&empty[s]), (lap - 1) & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
        break;
      }
      const int a = u / groups, k0 = (u - a * groups) * BK;
      const int boxes = (slots_of(a) + 15) / 16;  // of 16 slots (32 rows)
      const int e = expert[a], slot = base[a];
      if (elect_one()) {
        const uint32_t bar = smem_addr(&full[s]), at = sbase + (uint32_t)(s * stage_bytes);
        mbar_arrive_expect_tx(bar, (uint32_t)(kWTile + boxes * 32 * BK));
        tma_load_3d(at, &mapD, bar, k0, l0, e);
        for (int i = 0; i < boxes; ++i)
          tma_load_3d(at + kWTile + (uint32_t)(i * 32 * BK), &mapH, bar, k0, 2 * (slot + 16 * i), 0);
      }
      if (++s == p.down_stages) {
        s = 0;
        ++lap;
      }
    }
    for (int v = t > p.down_stages ? t - p.down_stages : 0; v < t; ++v)
      if (!poll_wait(smem_addr(&full[v % p.down_stages]), (uint32_t)(v / p.down_stages) & 1u, p.timeout_ns) && lane == 0)
        atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else if (warp == 1) {
    // a unit's two halves of 64 inner columns have scales, and so accumulators, of their own
    int issued = 0, done = 0, s = 0;
    uint32_t lap = 0;
    for (int t = 0; t < u1 - u0; ++t) {
      bool ok = poll_wait(smem_addr(&full[s]), lap & 1u, p.timeout_ns);
      const uint32_t idesc = moe_idesc(32 * ((slots_of((u0 + t) / groups) + 15) / 16));
      const uint32_t at = sbase + (uint32_t)(s * stage_bytes);
      const uint32_t wd = desc_lo(at), hd = desc_lo(at + kWTile);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        ok = ok && (t == 0 || poll_wait(smem_addr(&acc_empty[b]), (uint32_t)(t - 1) & 1u, p.timeout_ns));
        if (!ok) break;
        tmem_fence_after_sync();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            mma_f8(tmem + (uint32_t)(128 * b), make_desc(wd + (uint32_t)(2 * b + ks) * step_of(0)),
                   make_desc(hd + (uint32_t)(2 * b + ks) * step_of(0)), idesc, ks == 0 ? 0u : 1u);
          mma_commit(smem_addr(&acc_full[b]));
          if (b == 1) mma_commit(smem_addr(&empty[s]));
        }
        __syncwarp();
      }
      if (!ok) {
        if (elect_one()) mma_commit(smem_addr(&empty[s]));
        __syncwarp();
        issued = t + 1;
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        break;
      }
      issued = done = t + 1;
      if (++s == p.down_stages) {
        s = 0;
        ++lap;
      }
    }
    bool ok = true;  // every product has completed, and its commits have landed, before the CTA ends
    for (int u = issued > p.down_stages ? issued - p.down_stages : 0; u < issued; ++u)
      ok = ok && poll_wait(smem_addr(&empty[u % p.down_stages]), (uint32_t)(u / p.down_stages) & 1u, p.timeout_ns);
    for (int b = 0; b < 2 && done > 0; ++b)
      ok = ok && poll_wait(smem_addr(&acc_full[b]), (uint32_t)(done - 1) & 1u, p.timeout_ns);
    if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else {
    const int q = warp & 3;
    const int row = 32 * q + lane;
    const int fid = (int)threadIdx.x - 64;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
    float sum[kMoeMaxTokens];
#pragma unroll
    for (int j = 0; j < kMoeMaxTokens; ++j) sum[j] = 0.0f;
    bool ok = true;
    // scale of this thread's slot (fid < 64) in half v of the CTA's units, times the weights' scale
    const auto scale_of = [&](int v) {
      const int u = u0 + (v >> 1), a = u / groups, g = u - a * groups, hg = 2 * g + (v & 1);
      if (u >= u1 || fid >= slots_of(a) || hg >= p.h_groups) return 0.0f;
      return __ldg(p.sh + (int64_t)(base[a] + fid) * p.h_groups + hg) *
             __ldg(p.sd + (int64_t)expert[a] * p.stride_sd + (int64_t)(l0 >> 7) * p.ldsd + g);
    };
    const int halves = 2 * (u1 - u0);
    float s_next = fid < kMoeMaxTokens && halves > 0 ? scale_of(0) : 0.0f;
    for (int v = 0; v < halves; ++v) {
      const int b = v & 1, t = v >> 1;
      const int a = (u0 + t) / groups, n = slots_of(a);
      if (fid < kMoeMaxTokens) {
        col_scale[b][fid] = s_next;  // last read two halves ago: one barrier per half suffices
        s_next = scale_of(v + 1);
      }
      fold_barrier();
      if (ok) {  // a warp that gave up keeps meeting the others at the barrier
        ok = poll_wait(smem_addr(&acc_full[b]), (uint32_t)t & 1u, p.timeout_ns);
        if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
      }
      if (!ok) continue;
      tmem_fence_after_sync();
#pragma unroll
      for (int c = 0; c < kMoeMaxTokens / 8; ++c)
        if (8 * c < n) {
          float x[16];  // 8 slots: hi, lo, hi, lo, ...
          tmem_ld16(tq + (uint32_t)(128 * b + 16 * c), x);
          tmem_wait_ld();
          if (8 * (c + 1) >= n) {
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&acc_empty[b]));
          }
          tmem_ld_ready(x);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sum[8 * c + j] = fmaf(fmaf(x[2 * j + 1], 1.0f / kLoScale, x[2 * j]), col_scale[b][8 * c + j], sum[8 * c + j]);
        }
      if (b == 1 && (t + 1 == u1 - u0 || (u0 + t + 1) / groups != a)) {  // the expert's last unit here
#pragma unroll
        for (int j = 0; j < kMoeMaxTokens; ++j)
        {
          if (j < n) {
            float& y = ysum[slot_token[base[a] + j] * 128 + row];  // only this thread touches this row
            y = fmaf(slot_weight[base[a] + j], sum[j], y);
          }
          sum[j] = 0.0f;  // those past n too: they may hold what lay behind the expert's rows
        }
      }
    }
  }

  // ------------------------------------------------ the CTAs' sums, added in rank order
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, 256);
  __syncwarp();
  cluster_sync();
  const uint32_t y_addr = smem_addr(ysum);
  const int t0 = p.tokens * 128 * rank / p.split, t1 = p.tokens * 128 * (rank + 1) / p.split;
  for (int i = t0 + (int)threadIdx.x; i < t1; i += kThreads) {
    const int tok = i >> 7, col = l0 + (i & 127);
    float v = 0.0f;
    for (int r0 = 0; r0 < p.split; r0 += 8) {
      float u[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r0 + r < p.split)
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u[r]) : "r"(map_to_rank(y_addr + 4u * (uint32_t)i, (uint32_t)(r0 + r))) : "memory");
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r0 + r < p.split) v += u[r];
    }
    if (p.route.poisoned[tok]) v = __int_as_float(0x7FFFFFFF);
    if (col < p.hidden) {
      const int64_t o = (int64_t)tok * p.ldy + col;
      if (p.bf16) static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
      else        static_cast<float*>(p.y)[o] = v;
    }
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while a peer may read its sums
}

constexpr size_t kCtaSmem = 110 * 1024;  // two CTAs per SM
constexpr int kMaxSmem = 220 * 1024;

}  // namespace
}  // namespace f8

cudaError_t prepare_fp8_moe() {
  cudaError_t e = cudaFuncSetAttribute(f8::moe_up_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, f8::kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(f8::moe_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, f8::kMaxSmem);
  return e;
}

void shape_fp8_moe(MoeParams* p, int sm_count) {
  // as many stages as two CTAs per SM leave room for, two at least
  for (p->up_stages = f8::kMaxStages; p->up_stages > 2 && f8::up_smem(*p) > f8::kCtaSmem;) --p->up_stages;
  for (p->down_stages = f8::kMaxStages; p->down_stages > 2 && f8::down_smem(*p) > f8::kCtaSmem;) --p->down_stages;
  const int tiles = (p->hidden + 127) / 128;
  p->split = 1;
  while (p->split < 8 && tiles * p->split * 2 <= 2 * sm_count) p->split *= 2;
}

cudaError_t launch_fp8_moe(const MoeMaps& maps, const MoeParams& p, int sm_count, cudaStream_t stream) {
  const int col_tiles = (p.inner + f8::kUpCols - 1) / f8::kUpCols;
  const int grid = std::min(2 * sm_count, p.active_max * col_tiles);
  f8::moe_up_kernel<<<grid, f8::kThreads, f8::up_smem(p), stream>>>(maps.x, maps.gate, maps.up, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.hidden + 127) / 128 * p.split));
  cfg.blockDim = dim3(f8::kThreads);
  cfg.dynamicSmemBytes = f8::down_smem(p);
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
  return cudaLaunchKernelEx(&cfg, f8::moe_down_kernel, maps.h, maps.down, p);
}

}  // namespace sgemm_impl
