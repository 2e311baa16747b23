// kernel_fp8_moe.cu -- a mixture-of-experts layer for a few tokens on 8-bit weights, for sm_103a.
//
//     Y_t = sum_{e chosen by t} c_te W2_e (silu(W1_e x_t) * (W3_e x_t))
//
// Two kernels, both streams of the chosen experts' weights: every weight tile is loaded once and
// meets all the tokens that need it, as the 128 rows of a tensor-core product whose columns are
// tokens (16 to 64 of them, so the products cost little beside the loads).
//
// Every CTA of the first kernel works out the routing from the logits by itself (a warp per token),
// which costs less than a launch; the second kernel does too where it runs beside the first, and
// otherwise reads what the first left.
//
// moe_up_kernel takes tiles of 64 inner columns of active experts: rows 0-63 of the product are rows of
// W1_e, rows 64-127 rows of W3_e, the columns all the tokens in order, so x is loaded as it lies and no
// token is gathered.  The sums of the tokens that chose e become h = silu(gate) * up, stored as two
// E4M3 terms with a scale per 64 columns: hi = rn8(h / s), lo = rn8(16 (h / s - hi)), together within
// 2^-9.8 of the group's largest value.  As the second product is bound by the weights, the doubled
// columns are free.
//
// moe_down_kernel shares the (128 rows of the hidden side, expert, 128 inner columns) units evenly, in
// that order; a CTA folds its units per expert in FP32 registers and adds them weighted into its tokens'
// sums in shared memory.  Rows of one CTA go to Y; the others' sums go to slots of the workspace, and the
// last CTA of such rows to arrive adds them in CTA order (which CTA that is does not matter).  Unless there
// are many units per SM (shape_fp8_moe) a CTA of each kernel fits on an SM beside one of the other, and the
// second kernel is launched when the first has begun: it routes and fills its ring with W2 meanwhile, and
// waits for the first kernel only before it loads h (one token: 12 of its 17 MB of W2 are then on chip).
//
// Both: one CTA per SM with as many 16 KB weight tiles in flight as half its shared memory holds (all of it,
// where the kernels run one after the other); warp 0 loads (TMA), warp 1 issues the products, warp 2 loads
// scales a chunk of groups ahead, warps 4-7 fold the accumulators (several alternate) into FP32 sums in
// registers.
//
// What bounds it: up to 32 tokens the fold and the weights' bytes about equally, beyond that the fold.
// 32 tokens, 64 experts of 2048 x 1024, 8 each (397 MB): 98.6 us, 4.0 TB/s.  While it runs, the first kernel
// takes 820 cycles for a tile of 16 KB (5.8 TB/s at 1.9 GHz), of which the issuer waits 230 for an
// accumulator and 240 for operands; about 20 us are the routing, the first loads, the first kernel's part
// empty last round of tiles and the second's start and joining.  64 tokens: 132 us, 1050 cycles, 480 of them
// for an accumulator and 190 for operands.  One token (50 MB): 26 us, of which the launch, the routing, the
// first kernel's stream (9 us from its first wait to its last product), the wait between the kernels, the
// second stream and the last sums follow one another.
#include <algorithm>

#include "fp8_gemm.cuh"

namespace sgemm_impl {
namespace f8 {
namespace {

using namespace tc;

constexpr int BK = 128;
constexpr int kThreads = 256, kFirstFold = 4, kFoldWarps = 4, kFoldThreads = 128;
constexpr int kMaxStages = 10;
constexpr int kWTile = 128 * BK;  // 16 KB of weights per stage
constexpr int kUpCols = 64;       // inner columns of a tile of the first kernel
constexpr float kLoScale = 16.0f;
constexpr int kPitch = 129;
constexpr int kChunkGroups = 8;   // groups of 128 k whose scales are loaded together
constexpr int kChunks = 3;        // in shared memory

__device__ __forceinline__ void fold_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ uint32_t moe_idesc(int n) {  // E4M3, K-major, FP32 accumulator, M = 128
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// Total order of floats as unsigned integers; NaN is mapped to 0 (below -Inf) by the caller.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The routing, in shared memory: the experts that some token chose, in ascending order, each with its
// tokens, and a slot per (expert, token), numbered in that order.
struct Route {
  unsigned long long* mask_of;  // [experts] bit t: token t chose the expert
  unsigned long long* mask;     // [active] the same, of active experts
  int *expert, *base;           // [active] its number and first slot
  int* active_of;               // [experts]
  int* chosen;                  // [tokens][top_k] experts, -1: none
  float* weight;                // [tokens][top_k]
  int* slot_token;              // [slots]
  float* slot_weight;           // [slots]
  int* poisoned;                // [tokens] 1: a NaN or +Inf logit
  int* counts;                  // active experts, slots
};
__host__ __device__ inline size_t route_bytes(const MoeParams& p) {
  return 16 + (size_t)p.experts * 12 + (size_t)p.active_max * 16 + (size_t)p.slots_max * 16 + (size_t)p.tokens * 4;
}
__device__ __forceinline__ Route route_at(const MoeParams& p, void* smem) {
  Route r;
  r.mask_of = reinterpret_cast<unsigned long long*>((reinterpret_cast<uintptr_t>(smem) + 7) & ~uintptr_t(7));
  r.mask = r.mask_of + p.experts;
  r.expert = reinterpret_cast<int*>(r.mask + p.active_max);
  r.base = r.expert + p.active_max;
  r.active_of = r.base + p.active_max;
  r.chosen = r.active_of + p.experts;
  r.weight = reinterpret_cast<float*>(r.chosen + p.slots_max);
  r.slot_token = reinterpret_cast<int*>(r.weight + p.slots_max);
  r.slot_weight = reinterpret_cast<float*>(r.slot_token + p.slots_max);
  r.poisoned = reinterpret_cast<int*>(r.slot_weight + p.slots_max);
  r.counts = r.poisoned + p.tokens;
  return r;
}

// Dynamic shared memory, in this order: the ring of stages (1024-byte aligned), the scale chunks, the
// sums (first kernel: of an item's tokens; second: of Y), the routing.
__host__ __device__ inline int token_cols(const MoeParams& p) { return p.tokens <= 16 ? 16 : p.tokens <= 32 ? 32 : 64; }
__host__ __device__ inline size_t up_stage_bytes(const MoeParams& p) { return kWTile + (size_t)token_cols(p) * BK; }
__host__ __device__ inline int up_chunk_floats(const MoeParams& p) { return kChunkGroups * (token_cols(p) + 4); }
__host__ __device__ inline size_t up_smem(const MoeParams& p) {
  return 1024 + p.up_stages * up_stage_bytes(p) + (size_t)kChunks * up_chunk_floats(p) * 4 +
         (size_t)p.tokens * kPitch * 4 + route_bytes(p);
}
__host__ __device__ inline size_t down_stage_bytes(const MoeParams& p) {
  return kWTile + (size_t)2 * token_cols(p) * BK;
}
__host__ __device__ inline int down_chunk_floats(const MoeParams& p) {
  return 2 * kChunkGroups * token_cols(p) + kChunkGroups;
}
__host__ __device__ inline size_t down_smem(const MoeParams& p) {
  return 1024 + p.down_stages * down_stage_bytes(p) + (size_t)kChunks * down_chunk_floats(p) * 4 +
         (size_t)p.tokens * 128 * 4 + route_bytes(p);
}

// The logits of one token as a warp holds them: expert e = 32 i + lane has keys[i], 0 where it cannot
// be chosen (-Inf, past the end); returns whether one is NaN or +Inf.
template <int PER>
__device__ __forceinline__ bool load_keys(const MoeParams& p, int t, uint32_t (&keys)[PER]) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    keys[i] = 0u;
    if (32 * i + lane < p.experts) {
      const float x = get_at(p.guard, kSiteLogits, p.logits, (int64_t)t * p.ldl + 32 * i + lane, extent(p.tokens, p.ldl, p.experts));
      if (!(x < INFINITY)) bad = true;
      else if (x > -INFINITY) keys[i] = order_key(x + 0.0f);  // -0 counts as 0
    }
  }
  return bad;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// The warp's tokens t0, t0 + step, ...: their top_k experts with softmax weights to r.chosen and
// r.weight (expert -1 where there is none), 1 to r.poisoned for a token with a NaN or +Inf logit.
// PER: experts per lane at most.  top_k rounds of a warp maximum, TK tokens side by side: a round is
// 200 cycles of instructions that wait for one another.
template <int PER, int TK>
__device__ __forceinline__ void route_tokens(const MoeParams& p, const Route& r, int t0, int step) {
  const int lane = threadIdx.x & 31;
  for (; t0 < p.tokens; t0 += TK * step) {
    uint32_t keys[TK][PER];
    bool bad[TK];
#pragma unroll
    for (int q = 0; q < TK; ++q) {
#pragma unroll
      for (int i = 0; i < PER; ++i) keys[q][i] = 0u;
      bad[q] = false;
      if (t0 + q * step < p.tokens) bad[q] = load_keys(p, t0 + q * step, keys[q]);
    }
    uint32_t most[TK], mine[TK];  // lane j: choice j
    int mine_e[TK];
    float all[TK];
#pragma unroll
    for (int q = 0; q < TK; ++q) {
      bad[q] = __any_sync(0xffffffffu, bad[q]);
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (bad[q]) keys[q][i] = 0u;  // nothing is chosen
        m = max(m, keys[q][i]);
      }
      most[q] = __reduce_max_sync(0xffffffffu, m);
      all[q] = 0.0f;
      mine[q] = 0u;
      mine_e[q] = -1;
    }
    if (!p.renormalize)  // over all experts
#pragma unroll
      for (int q = 0; q < TK; ++q) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (keys[q][i] != 0u) all[q] += expf(key_value(keys[q][i]) - key_value(most[q]));
        all[q] = warp_sum(all[q]);
      }
    for (int j = 0; j < p.top_k; ++j) {
#pragma unroll
      for (int q = 0; q < TK; ++q) {
        uint32_t best = keys[q][0];
#pragma unroll
        for (int i = 1; i < PER; ++i) best = max(best, keys[q][i]);
        const uint32_t k = __reduce_max_sync(0xffffffffu, best);
        int e = -1;  // ties: the lowest index
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
          const unsigned at = __ballot_sync(0xffffffffu, keys[q][i] == k);
          if (at != 0u) e = 32 * i + __ffs((int)at) - 1;
        }
        if (k == 0u) e = -1;  // no expert that can be chosen is left
        if (lane == j) {
          mine[q] = k;
          mine_e[q] = e;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (e == 32 * i + lane) keys[q][i] = 0u;
      }
    }
#pragma unroll
    for (int q = 0; q < TK; ++q) {
      const int t = t0 + q * step;
      const float w = mine_e[q] >= 0 ? expf(key_value(mine[q]) - key_value(most[q])) : 0.0f;
      const float sum = p.renormalize ? warp_sum(w) : all[q];
      if (t >= p.tokens) continue;
      if (lane == 0) r.poisoned[t] = bad[q] ? 1 : 0;
      if (lane < p.top_k) {
        r.chosen[t * p.top_k + lane] = mine_e[q];
        r.weight[t * p.top_k + lane] = w / sum;
      }
    }
  }
}

// The whole routing by the CTA's threads.
__device__ __forceinline__ void route(const MoeParams& p, const Route& r) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = (int)threadIdx.x; e < p.experts; e += kThreads) r.mask_of[e] = 0ull;
  if (p.experts <= 64 && p.tokens <= kThreads / 32) route_tokens<2, 1>(p, r, warp, kThreads / 32);
  else if (p.experts <= 64) route_tokens<2, 4>(p, r, warp, kThreads / 32);
  else if (p.experts <= 128) route_tokens<4, 4>(p, r, warp, kThreads / 32);
  else if (p.experts <= 256) route_tokens<8, 2>(p, r, warp, kThreads / 32);
  else route_tokens<kMoeMaxExperts / 32, 1>(p, r, warp, kThreads / 32);
  __syncthreads();
  for (int i = (int)threadIdx.x; i < p.slots_max; i += kThreads)
    if (r.chosen[i] >= 0) {
      const int t = i / p.top_k;
      atomicOr(reinterpret_cast<unsigned*>(&r.mask_of[r.chosen[i]]) + (t >> 5), 1u << (t & 31));
    }
  __syncthreads();
  if (warp == 0) {  // 32 experts at a time
    int n = 0, slots = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + lane;
      const unsigned long long m = e < p.experts ? r.mask_of[e] : 0ull;
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
        r.active_of[e] = a;
      }
      n += __popc(act);
      slots += __shfl_sync(0xffffffffu, before, 31);
    }
    if (lane == 0) {
      r.counts[0] = n;
      r.counts[1] = slots;
    }
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < p.slots_max; i += kThreads)
    if (r.chosen[i] >= 0) {
      const int t = i / p.top_k, a = r.active_of[r.chosen[i]];
      const int slot = r.base[a] + __popcll(r.mask[a] & ((1ull << t) - 1ull));
      r.slot_token[slot] = t;
      r.slot_weight[slot] = r.weight[i];
    }
  __syncthreads();
}

__device__ __forceinline__ int64_t route_words(const MoeParams& p) {
  return 2 + 2 * (int64_t)p.active_max + 2 * (int64_t)p.slots_max + p.tokens;
}

// What the second kernel needs of it, to (store) or from the workspace, by `threads` threads.
__device__ __forceinline__ void copy_route(const MoeParams& p, const Route& r, bool store, int thread, int threads) {
  const auto copy = [&](int* shared, int* global, int n) {
    for (int i = thread; i < n; i += threads) {
      if (!in_range(p.guard.fault, p.guard.word, kSitePart, global + i - p.route, 1, route_words(p))) continue;
      if (store) global[i] = shared[i];
      else       shared[i] = global[i];
    }
  };
  int* g = p.route;
  copy(r.counts, g, 2);
  copy(r.expert, g += 2, p.active_max);
  copy(r.base, g += p.active_max, p.active_max);
  copy(r.slot_token, g += p.active_max, p.slots_max);
  copy(reinterpret_cast<int*>(r.slot_weight), g += p.slots_max, p.slots_max);
  copy(r.poisoned, g + p.slots_max, p.tokens);
}

// Scales that stored matrices of `rows` rows and `groups` groups of columns have, all experts'.
__device__ __forceinline__ int64_t expert_scales(int experts, int64_t stride, int rows, int64_t ld, int groups) {
  return (experts - 1) * stride + extent((rows + 127) / 128, ld, groups);
}

// NC: columns of the product, the tokens rounded up to 16, 32 or 64.
template <int NC>
__global__ void __launch_bounds__(kThreads, 2) moe_up_kernel(const __grid_constant__ CUtensorMap mapX,
                                                             const __grid_constant__ CUtensorMap mapG,
                                                             const __grid_constant__ CUtensorMap mapU,
                                                             const __grid_constant__ MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], done[kMaxStages];
  // accumulators: as many as 128 columns hold, so that products and loads go on while an item's sums are
  // worked into h; no more than stages, as a stage's second commit must not precede the folders' look at
  // its first
  constexpr int kBufs = 128 / NC;
  const int bufs = kBufs <= 2 ? kBufs : min(kBufs, p.up_stages);  // (there are 2 stages at least)
  __shared__ __align__(8) uint64_t acc_empty[kBufs];
  __shared__ __align__(8) uint64_t scale_full[kChunks], scale_empty[kChunks];
  __shared__ uint32_t tmem_slot;

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  constexpr int stage_bytes = kWTile + NC * BK;
  constexpr int kChunkFloats = kChunkGroups * (NC + 4);  // per group: NC token scales, gate's, up's
  float* chunks = reinterpret_cast<float*>(smem_raw + pad + p.up_stages * stage_bytes);
  float* sums = chunks + kChunks * kChunkFloats;  // [slot of the expert][kPitch]
  const Route r = route_at(p, sums + p.tokens * kPitch);
  const int col_tiles = (p.inner + kUpCols - 1) / kUpCols;
  const int groups = (p.hidden + BK - 1) / BK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tensormap(&mapX);
    prefetch_tensormap(&mapG);
    prefetch_tensormap(&mapU);
    for (int s = 0; s < p.up_stages; ++s) {
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
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), 128);
  // what the stream's kernel before this one wrote; the second kernel may begin once that is there
  // too, as it reads the logits on its own
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tmem_fence_before_sync();
  route(p, r);
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (blockIdx.x == gridDim.x - 1 && warp == 3) {  // by a warp with nothing else to do
    for (int i = lane; i < (p.hidden + 127) / 128; i += 32) put_at(p.guard, kSitePart, p.arrived, i, (p.hidden + 127) / 128, 0);
    if (p.many) copy_route(p, r, true, lane, 32);
  }
  const int items = r.counts[0] * col_tiles;
  const int my_items = (int)blockIdx.x < items ? (items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;

  if (warp == 0) {
    int t = 0, s = 0;
    uint32_t lap = 0;
    bool ok = true;
    for (int i = 0; ok && i < my_items; ++i) {
      const int item = (int)blockIdx.x + i * (int)gridDim.x;
      const int e = r.expert[item / col_tiles], c0 = (item % col_tiles) * kUpCols;
      for (int g = 0; g < groups; ++g, ++t) {
        if (lap > 0 && !poll_wait(smem_addr(&done[s]), (lap - 1) & 1u, p.timeout_ns)) {
          if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t bar = smem_addr(&full[s]), a = sbase + (uint32_t)(s * stage_bytes);
          mbar_arrive_expect_tx(bar, (uint32_t)stage_bytes);
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
    constexpr uint32_t step = 32u >> 4;
    const uint32_t desc0 = desc_lo(sbase);
    const int units = my_items * groups;
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
        const uint32_t wd = desc0 + (uint32_t)(s * (stage_bytes >> 4)), xd = wd + (kWTile >> 4);
#pragma unroll
        for (uint32_t ks = 0; ks < BK / 32; ++ks)
          mma_f8(tmem + (uint32_t)(b * NC), make_desc(wd + ks * step), make_desc(xd + ks * step), moe_idesc(NC),
                 ks == 0 ? 0u : 1u);
        mma_commit(smem_addr(&done[s]));  // the stage is free, the accumulator holds group t
      }
      __syncwarp();
      if (++b == bufs) {
        b = 0;
        ++b_lap;
      }
      if (++s == p.up_stages) {
        s = 0;
        ++lap;
      }
    }
    bool ok = true;  // every product has completed, and its commit has landed, before the CTA ends
    for (int u = t > p.up_stages ? t - p.up_stages : 0; u < t; ++u)
      ok = ok && poll_wait(smem_addr(&done[u % p.up_stages]), (uint32_t)(u / p.up_stages) & 1u, p.timeout_ns);
    if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else if (warp == 2) {
    const uint32_t ring = smem_addr(chunks);
    int c = 0;
    uint32_t lap = 0;
    bool ok = true;
    for (int i = 0; ok && i < my_items; ++i) {
      const int item = (int)blockIdx.x + i * (int)gridDim.x;
      const int e = r.expert[item / col_tiles], rb = (item % col_tiles) * kUpCols >> 7;
      const int64_t sg = (int64_t)e * p.stride_sg + (int64_t)rb * p.ldsg, su = (int64_t)e * p.stride_su + (int64_t)rb * p.ldsu;
      for (int g0 = 0; g0 < groups; g0 += kChunkGroups) {
        if (lap > 0 && !poll_wait(smem_addr(&scale_empty[c]), (lap - 1) & 1u, p.timeout_ns)) {
          if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
          ok = false;
          break;
        }
        const uint32_t dst = ring + 4u * (uint32_t)(c * kChunkFloats);
        const int count = min(kChunkGroups, groups - g0);
        for (int j = lane; j < NC + 2; j += 32) {
          const float* src = j < NC ? p.sx : j == NC ? p.sg : p.su;
          const int64_t at = (j < NC ? (int64_t)min(j, p.tokens - 1) * p.ldsx : j == NC ? sg : su) + g0;
          const int64_t n = j < NC    ? extent(p.tokens, p.ldsx, groups)
                            : j == NC ? expert_scales(p.experts, p.stride_sg, p.inner, p.ldsg, groups)
                                      : expert_scales(p.experts, p.stride_su, p.inner, p.ldsu, groups);
          for (int g = 0; g < count; ++g)
            copy4_async(p.guard, kSiteScale, dst + 4u * (uint32_t)(g * (NC + 4) + j), src, at + g, n);
        }
        copies_arrive(smem_addr(&scale_full[c]));
        if (++c == kChunks) {
          c = 0;
          ++lap;
        }
      }
    }
    copies_wait_all();
  } else if (warp >= kFirstFold) {
    const int q = warp & 3;
    const int row = 32 * q + lane;  // rows 0-63: gate, 64-127: up
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
    bool ok = true;
    int s = 0, c = 0, b = 0;
    uint32_t s_lap = 0, c_lap = 0;
    for (int i = 0; i < my_items; ++i) {
      const int item = (int)blockIdx.x + i * (int)gridDim.x;
      const int a = item / col_tiles, c0 = (item % col_tiles) * kUpCols;
      float2 sum[NC / 2];
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) sum[j] = make_float2(0.0f, 0.0f);
      for (int g = 0; ok && g < groups; ++g) {
        const int in_chunk = g & (kChunkGroups - 1);
        if (in_chunk == 0) ok = poll_wait(smem_addr(&scale_full[c]), c_lap & 1u, p.timeout_ns);
        ok = ok && poll_wait(smem_addr(&done[s]), s_lap & 1u, p.timeout_ns);
        if (!ok) {
          if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
          break;
        }
        tmem_fence_after_sync();
        const float* sc = chunks + c * kChunkFloats + in_chunk * (NC + 4);
        const float w = sc[NC + (q >> 1)];
        const float2 w2 = make_float2(w, w);
#pragma unroll
        for (int j0 = 0; j0 < NC; j0 += 32) {
          constexpr int kCols = NC < 32 ? NC : 32;
          float v[kCols];
          tmem_ld(tq + (uint32_t)(b * NC + j0), v);
          tmem_wait_ld();
          if (j0 + kCols == NC) {
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&acc_empty[b]));
          }
#pragma unroll
          for (int j = 0; j < kCols; ++j) asm volatile("" : "+f"(v[j]));  // used behind the wait only
#pragma unroll
          for (int j = 0; j < kCols; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(sc + j0 + j);
            float2* m = &sum[(j0 + j) / 2];
            // the two scales first: either alone may be far from 1
            m[0] = __ffma2_rn(make_float2(v[j], v[j + 1]), __fmul2_rn(make_float2(x.x, x.y), w2), m[0]);
            m[1] = __ffma2_rn(make_float2(v[j + 2], v[j + 3]), __fmul2_rn(make_float2(x.z, x.w), w2), m[1]);
          }
        }
        if (in_chunk == kChunkGroups - 1 || g == groups - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&scale_empty[c]));
          if (++c == kChunks) {
            c = 0;
            ++c_lap;
          }
        }
        if (++b == bufs) b = 0;
        if (++s == p.up_stages) {
          s = 0;
          ++s_lap;
        }
      }
      // the chosen tokens' sums, compacted, to shared memory; then a warp per slot.  (A warp that gave
      // up keeps meeting the others at the barriers.)
      const unsigned long long mask = r.mask[a];
      fold_barrier();  // the previous item's sums have been read
      {
        int at = row;
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if ((mask >> j) & 1ull) {
            sums[at] = j & 1 ? sum[j / 2].y : sum[j / 2].x;
            at += kPitch;
          }
      }
      fold_barrier();
      if (!ok) continue;
      const int n = __popcll(mask);
      for (int j = warp - kFirstFold; j < n; j += kFoldWarps) {
        const float* u = sums + j * kPitch;
        float h[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float gate = u[2 * lane + k], up = u[64 + 2 * lane + k];
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
          uint16_t* pairs = reinterpret_cast<uint16_t*>(p.h);
          const int64_t n = (int64_t)p.slots_max * p.inner;
          const int64_t at = slot * p.inner + (col >> 1);
          put_at(p.guard, kSitePart, pairs, at, n, (uint16_t)hi);
          put_at(p.guard, kSitePart, pairs, at + (p.inner >> 1), n, (uint16_t)lo);
        }
        if (lane == 0)
          put_at(p.guard, kSitePart, p.sh, slot * p.h_groups + c0 / kUpCols, (int64_t)p.slots_max * p.h_groups, scale);
      }
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, 128);
}

__device__ __forceinline__ int64_t part_words(const MoeParams& p) { return 2 * (int64_t)p.down_grid * p.tokens * 128; }

__device__ __forceinline__ void store_y(const MoeParams& p, int tok, int col, int poisoned, float v) {
  if (col >= p.hidden) return;
  if (poisoned) v = __int_as_float(0x7FFFFFFF);
  const int64_t o = (int64_t)tok * p.ldy + col;
  if (!in_range(p.guard.fault, p.guard.word, kSiteOut, o, 1, extent(p.tokens, p.ldy, p.hidden))) return;
  if (p.bf16) static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
  else        static_cast<float*>(p.y)[o] = v;
}

// NC: the tokens rounded up to 16, 32 or 64: slots of an expert at most.
template <int NC>
__global__ void __launch_bounds__(kThreads, 2) moe_down_kernel(const __grid_constant__ CUtensorMap mapH,
                                                               const __grid_constant__ CUtensorMap mapD,
                                                               const __grid_constant__ MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], done[kMaxStages];
  __shared__ __align__(8) uint64_t scale_full[kChunks], scale_empty[kChunks];
  __shared__ uint32_t tmem_slot;
  __shared__ int last_tiles[2], n_last;  // tiles whose last sums are this CTA's (of two that it shares at most)

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  constexpr int stage_bytes = kWTile + 2 * NC * BK;
  constexpr int kChunkFloats = 2 * kChunkGroups * NC + kChunkGroups;  // slots' scales of 16 halves, weights' of 8 units
  constexpr uint32_t kHalfCols = 2 * NC, kAccCols = 4 * NC;           // of an accumulator: a unit's two halves
  constexpr uint32_t kTmemCols = 256;               // 128 of an SM's 512 are the first kernel's
  constexpr int kBufs = kTmemCols / kAccCols;
  const int bufs = kBufs <= 2 ? kBufs : min(kBufs, p.down_stages);  // as in the first kernel
  __shared__ __align__(8) uint64_t acc_empty[kBufs];
  float* chunks = reinterpret_cast<float*>(smem_raw + pad + p.down_stages * stage_bytes);
  float* ysum = chunks + kChunks * kChunkFloats;  // [tokens][128]
  const Route r = route_at(p, ysum + p.tokens * 128);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (p.hidden + 127) / 128;  // of rows
  const int groups = (p.inner + BK - 1) / BK;

  if (threadIdx.x == 0) {
    n_last = 0;
    prefetch_tensormap(&mapH);
    prefetch_tensormap(&mapD);
    for (int s = 0; s < p.down_stages; ++s) {
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
  for (int i = (int)threadIdx.x; i < p.tokens * 128; i += kThreads) ysum[i] = 0.0f;
  tmem_fence_before_sync();
  if (p.many) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    copy_route(p, r, false, (int)threadIdx.x, kThreads);
    __syncthreads();
  } else {
    route(p, r);  // the logits were complete before the first kernel let this one begin
  }
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const int n_active = r.counts[0], n_slots = r.counts[1];
  const int *expert = r.expert, *base = r.base;
  // this CTA's units: [u0, u0 + mine) of tiles x active experts x groups
  const int64_t per_tile = (int64_t)n_active * groups, total = per_tile * tiles;
  const int ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, total));  // that have units: one at least each
  const auto bound = [&](int c) { return total * min(c, ctas) / ctas; };
  const int64_t u0 = bound((int)blockIdx.x);
  const int mine = (int)(bound((int)blockIdx.x + 1) - u0);
  struct Place {  // of a unit: row tile, active expert, group
    int tile, a, g;
  };
  const Place first = {per_tile > 0 ? (int)(u0 / per_tile) : 0, per_tile > 0 ? (int)(u0 % per_tile) / groups : 0,
                       per_tile > 0 ? (int)(u0 % per_tile) % groups : 0};
  const auto next = [&](Place* u) {
    if (++u->g == groups) {
      u->g = 0;
      if (++u->a == n_active) {
        u->a = 0;
        ++u->tile;
      }
    }
  };
  const auto slots_of = [&](int a) { return (a + 1 < n_active ? base[a + 1] : n_slots) - base[a]; };

  if (warp == 0) {
    // the weights of the first units while the first kernel runs, their inner values when it is done
    const int ahead = min(p.down_stages, mine);
    const auto load = [&](int s, const Place& u, bool weights, bool inner) {
      const int boxes = (slots_of(u.a) + 15) / 16;  // of 16 slots (32 rows)
      const int e = expert[u.a], slot = base[u.a];
      if (elect_one()) {
        const uint32_t bar = smem_addr(&full[s]), at = sbase + (uint32_t)(s * stage_bytes);
        if (weights) {
          mbar_arrive_expect_tx(bar, (uint32_t)(kWTile + boxes * 32 * BK));
          tma_load_3d(at, &mapD, bar, u.g * BK, u.tile * 128, e);
        }
        if (inner)
          for (int i = 0; i < boxes; ++i)
            tma_load_3d(at + kWTile + (uint32_t)(i * 32 * BK), &mapH, bar, u.g * BK, 2 * (slot + 16 * i), 0);
      }
      __syncwarp();
    };
    Place u = first;
    if (!p.many)
      for (int t = 0; t < ahead; ++t, next(&u)) load(t, u, true, false);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    u = first;
    for (int t = 0; t < ahead; ++t, next(&u)) load(t, u, p.many != 0, true);
    int t = ahead, s = 0;
    uint32_t lap = 1;
    for (; t < mine; ++t, next(&u)) {
      if (!poll_wait(smem_addr(&done[s]), (lap - 1) & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
        break;
      }
      load(s, u, true, true);
      if (++s == p.down_stages) {
        s = 0;
        ++lap;
      }
    }
    for (int v = t > p.down_stages ? t - p.down_stages : 0; v < t; ++v)
      if (!poll_wait(smem_addr(&full[v % p.down_stages]), (uint32_t)(v / p.down_stages) & 1u, p.timeout_ns) && lane == 0)
        atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else if (warp == 1) {
    // a unit's two halves of 64 inner columns have scales, and so columns of the accumulator, of their own
    constexpr uint32_t step = 32u >> 4;
    const uint32_t desc0 = desc_lo(sbase);
    int t = 0, s = 0, b = 0;
    Place u = first;
    uint32_t lap = 0, b_lap = 0;
    for (; t < mine; ++t, next(&u)) {
      if ((b_lap > 0 && !poll_wait(smem_addr(&acc_empty[b]), (b_lap - 1) & 1u, p.timeout_ns)) ||
          !poll_wait(smem_addr(&full[s]), lap & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        break;
      }
      const uint32_t idesc = moe_idesc(32 * ((slots_of(u.a) + 15) / 16));
      tmem_fence_after_sync();
      if (elect_one()) {
        const uint32_t wd = desc0 + (uint32_t)(s * (stage_bytes >> 4)), hd = wd + (kWTile >> 4);
        const uint32_t acc = tmem + (uint32_t)b * kAccCols;
#pragma unroll
        for (uint32_t ks = 0; ks < 4; ++ks)
          mma_f8(acc + (ks >> 1) * kHalfCols, make_desc(wd + ks * step), make_desc(hd + ks * step), idesc, ks & 1u);
        mma_commit(smem_addr(&done[s]));  // the stage is free, the accumulator holds unit t
      }
      __syncwarp();
      if (++b == bufs) {
        b = 0;
        ++b_lap;
      }
      if (++s == p.down_stages) {
        s = 0;
        ++lap;
      }
    }
    bool ok = true;  // every product has completed, and its commit has landed, before the CTA ends
    for (int u = t > p.down_stages ? t - p.down_stages : 0; u < t; ++u)
      ok = ok && poll_wait(smem_addr(&done[u % p.down_stages]), (uint32_t)(u / p.down_stages) & 1u, p.timeout_ns);
    if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  } else if (warp == 2) {
    // chunks: up to 8 consecutive units of one expert
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t ring = smem_addr(chunks);
    int c = 0;
    Place u = first;
    uint32_t lap = 0;
    for (int t = 0; t < mine;) {
      if (lap > 0 && !poll_wait(smem_addr(&scale_empty[c]), (lap - 1) & 1u, p.timeout_ns)) {
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
        break;
      }
      const int count = min(min(kChunkGroups, groups - u.g), mine - t);
      const uint32_t dst = ring + 4u * (uint32_t)(c * kChunkFloats);
      const int n = slots_of(u.a), halves = min(2 * count, p.h_groups - 2 * u.g);
      for (int j = lane; j < n; j += 32) {
        const int64_t src = (int64_t)(base[u.a] + j) * p.h_groups + 2 * u.g;
        for (int h = 0; h < halves; ++h)
          copy4_async(p.guard, kSitePart, dst + 4u * (uint32_t)(h * NC + j), p.sh, src + h, (int64_t)p.slots_max * p.h_groups);
      }
      if (lane < count)
        copy4_async(p.guard, kSiteScale, dst + 4u * (uint32_t)(2 * kChunkGroups * NC + lane), p.sd,
                    (int64_t)expert[u.a] * p.stride_sd + (int64_t)u.tile * p.ldsd + u.g + lane,
                    expert_scales(p.experts, p.stride_sd, p.hidden, p.ldsd, groups));
      copies_arrive(smem_addr(&scale_full[c]));
      t += count;
      u.g += count - 1;
      next(&u);
      if (++c == kChunks) {
        c = 0;
        ++lap;
      }
    }
    copies_wait_all();
  } else if (warp >= kFirstFold) {
    const int q = warp & 3;
    const int row = 32 * q + lane;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
    float sum[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) sum[j] = 0.0f;
    bool ok = true;
    int s = 0, c = 0, b = 0;
    Place u = first;
    uint32_t s_lap = 0, c_lap = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters of arrivals are the first kernel's
    if (total == 0)  // no token chose anything
      for (int tile = (int)blockIdx.x; tile < tiles; tile += (int)gridDim.x)
        for (int t = 0; t < p.tokens; ++t) store_y(p, t, tile * 128 + row, r.poisoned[t], 0.0f);
    for (int t = 0; t < mine;) {
      // a chunk of units of one expert, whose slots are rounded up to NS (with their number at run time
      // the fold took 1400 cycles a unit)
      const int count = min(min(kChunkGroups, groups - u.g), mine - t), n = slots_of(u.a);
      ok = ok && poll_wait(smem_addr(&scale_full[c]), c_lap & 1u, p.timeout_ns);
      const bool flush = t + count == mine || u.g + count == groups;  // the expert's last units here
      const auto run = [&](auto slots) {
        constexpr int NS = decltype(slots)::value;
        const float* sc = chunks + c * kChunkFloats;
        for (int i = 0; ok && i < count; ++i, sc += 2 * NC) {
          ok = poll_wait(smem_addr(&done[s]), s_lap & 1u, p.timeout_ns);
          if (!ok) break;
          tmem_fence_after_sync();
          const uint32_t acc = tq + (uint32_t)b * kAccCols;
          const float w = chunks[c * kChunkFloats + 2 * kChunkGroups * NC + i];
          const bool two = 2 * (u.g + i) + 1 < p.h_groups;  // the second half may be past the end, its scales not loaded
#pragma unroll
          for (int j0 = 0; j0 < NS; j0 += 8) {  // 8 slots of both halves: hi, lo, hi, lo, ...
            float x[2][16];
            tmem_ld16(acc + (uint32_t)(2 * j0), x[0]);
            tmem_ld16(acc + kHalfCols + (uint32_t)(2 * j0), x[1]);
            float4 f[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              f[0][k] = *reinterpret_cast<const float4*>(sc + j0 + 4 * k);
              f[1][k] = *reinterpret_cast<const float4*>(sc + NC + j0 + 4 * k);
            }
            tmem_wait_ld();
            if (j0 + 8 == NS) {
              tmem_fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&acc_empty[b]));
            }
            tmem_ld_ready(x[0]);
            tmem_ld_ready(x[1]);
            const float f0[8] = {f[0][0].x, f[0][0].y, f[0][0].z, f[0][0].w, f[0][1].x, f[0][1].y, f[0][1].z, f[0][1].w};
            const float f1[8] = {f[1][0].x, f[1][0].y, f[1][0].z, f[1][0].w, f[1][1].x, f[1][1].y, f[1][1].z, f[1][1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float v0 = fmaf(x[0][2 * j + 1], 1.0f / kLoScale, x[0][2 * j]);
              const float v1 = fmaf(x[1][2 * j + 1], 1.0f / kLoScale, x[1][2 * j]);
              sum[j0 + j] = fmaf(v0, f0[j] * w, sum[j0 + j]);
              if (two) sum[j0 + j] = fmaf(v1, f1[j] * w, sum[j0 + j]);
            }
          }
          if (++b == bufs) b = 0;
          if (++s == p.down_stages) {
            s = 0;
            ++s_lap;
          }
        }
        if (flush) {
          const int slot = base[u.a];
#pragma unroll
          for (int j0 = 0; j0 < NS; j0 += 8) {
            float* y[8];
            float v[8], cw[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const bool in = j0 + j < n;
              y[j] = &ysum[(in ? r.slot_token[slot + j0 + j] : 0) * 128 + row];  // only this thread touches this row
              cw[j] = in ? r.slot_weight[slot + j0 + j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = *y[j];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (j0 + j < n) *y[j] = fmaf(cw[j], sum[j0 + j], v[j]);  // an expert's tokens differ
              sum[j0 + j] = 0.0f;  // those past n too: they may hold what lay behind the expert's rows
            }
          }
        }
      };
      if (n <= 8) run(std::integral_constant<int, 8>{});
      else if (n <= 16) run(std::integral_constant<int, 16>{});
      else if (NC >= 32 && n <= 32) run(std::integral_constant<int, NC >= 32 ? 32 : 16>{});
      else run(std::integral_constant<int, NC>{});
      if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);  // (the barriers below are met all the same)
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&scale_empty[c]));
      if (++c == kChunks) {
        c = 0;
        ++c_lap;
      }
      t += count;
      u.g += count - 1;
      const Place at = u;
      next(&u);
      const bool end = t == mine;
      if (end || u.tile != at.tile) {  // the tile's last unit here: Y, or a slot
        const int64_t t0 = at.tile * per_tile, t1 = t0 + per_tile;
        const int col = at.tile * 128 + row;
        if (u0 <= t0 && u0 + mine >= t1) {
          for (int tok = 0; tok < p.tokens; ++tok) store_y(p, tok, col, r.poisoned[tok], ysum[tok * 128 + row]);
        } else {
          // CTAs c0 .. c1 share the tile; one that began before it uses its first slot for it, one that began
          // in it its second
          const int c0 = (int)(((t0 + 1) * ctas + total - 1) / total - 1), c1 = (int)((t1 * ctas + total - 1) / total - 1);
          const int64_t to = (2 * (int64_t)blockIdx.x + (u0 < t0 ? 0 : 1)) * p.tokens * 128 + row;
          for (int tok = 0; tok < p.tokens; ++tok)
            put_at(p.guard, kSitePart, p.part, to + tok * 128, part_words(p), ysum[tok * 128 + row]);
          __threadfence();
          fold_barrier();
          if (threadIdx.x == kFirstFold * 32 && in_range(p.guard.fault, p.guard.word, kSitePart, at.tile, 1, tiles) && atomicAdd(&p.arrived[at.tile], 1) == c1 - c0)
            last_tiles[n_last++] = at.tile;  // the others' sums are there
        }
        for (int tok = 0; tok < p.tokens; ++tok) ysum[tok * 128 + row] = 0.0f;
      }
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);

  // ------------------------------------------------ the slots of such tiles, added in CTA order: a warp
  // per token, four rows a lane, the loads of eight slots of two tokens in flight
  for (int i = 0; i < n_last; ++i) {
    __threadfence();
    const int tile = last_tiles[i];
    const int64_t t0 = tile * per_tile, t1 = t0 + per_tile;
    const int c0 = (int)(((t0 + 1) * ctas + total - 1) / total - 1), c1 = (int)((t1 * ctas + total - 1) / total - 1);
    const int64_t slot = (int64_t)p.tokens * 128;
    const int64_t from = (2 * (int64_t)c0 + 1) * slot + 4 * lane;
    const int64_t back = bound(c0) < t0 ? -slot : 0;  // only c0 can have begun before the tile
    for (int tok0 = warp; tok0 < p.tokens; tok0 += 2 * (kThreads / 32)) {
      float4 v[2];
      v[0] = v[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k0 = 0; k0 <= c1 - c0; k0 += 8) {
        float4 x[2][8];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int tok = tok0 + q * (kThreads / 32);
            x[q][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const int64_t word = from + 2 * (k0 + k) * slot + (k0 + k == 0 ? back : 0) + tok * 128;
            if (k0 + k <= c1 - c0 && tok < p.tokens && in_range(p.guard.fault, p.guard.word, kSitePart, word, 4, part_words(p)))
              x[q][k] = __ldcg(reinterpret_cast<const float4*>(p.part + word));
          }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            v[q].x += x[q][k].x;
            v[q].y += x[q][k].y;
            v[q].z += x[q][k].z;
            v[q].w += x[q][k].w;
          }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int tok = tok0 + q * (kThreads / 32), col = tile * 128 + 4 * lane;
        if (tok >= p.tokens) continue;
        store_y(p, tok, col, r.poisoned[tok], v[q].x);
        store_y(p, tok, col + 1, r.poisoned[tok], v[q].y);
        store_y(p, tok, col + 2, r.poisoned[tok], v[q].z);
        store_y(p, tok, col + 3, r.poisoned[tok], v[q].w);
      }
    }
  }
}

constexpr size_t kHalfSmem = 112 * 1024;  // a CTA of each kernel per SM
constexpr size_t kMaxSmem = 222 * 1024;

// f(NC) for the token columns of p.
template <typename F>
cudaError_t with_token_cols(int cols, const F& f) {
  return cols == 16   ? f(std::integral_constant<int, 16>{})
         : cols == 32 ? f(std::integral_constant<int, 32>{})
                      : f(std::integral_constant<int, 64>{});
}

cudaError_t launch_pdl(const void* kernel, int grid, size_t smem, void** args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace
}  // namespace f8

cudaError_t prepare_fp8_moe() {
  for (int cols = 16; cols <= 64; cols *= 2) {
    const cudaError_t e = f8::with_token_cols(cols, [](auto nc) {
      constexpr int NC = decltype(nc)::value;
      cudaError_t err = cudaSuccess;
      for (const void* kernel : {reinterpret_cast<const void*>(f8::moe_up_kernel<NC>),
                                 reinterpret_cast<const void*>(f8::moe_down_kernel<NC>)}) {
        if (err == cudaSuccess)
          err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)f8::kMaxSmem);
        // all of the SM's memory, so that the second kernel's CTAs find room beside the first's
        if (err == cudaSuccess)
          err = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
      }
      return err;
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

void shape_fp8_moe(MoeParams* p, int sm_count) {
  const int64_t units = (int64_t)p->active_max * ((p->inner + 127) / 128) * ((p->hidden + 127) / 128);
  p->down_grid = (int)std::min<int64_t>(sm_count, units);
  // Half the shared memory each, so that the second kernel routes and fills its ring while the first runs, or
  // all of it for one after the other, whose bytes in flight pay where there are many units per SM, the sooner
  // the more tokens' inner values a stage holds.  Measured over 90 layers (us beside / after, at units per SM):
  //   16 columns:  13.5 38.8 / 44.8,  54 83.5 / 87.9,  81 110.8 / 110.9,  162 143 / 145,  216 254 / 244
  //   32 columns:  13.5 47.5 / 52.0,  54 98.5 / 101.6,  61 105.6 / 106.4,  81 135.9 / 132.2,  108 165.9 / 159.0
  //   64 columns:  10 53.3 / 57.7,  20 70.8 / 73.4 and 82.5 / 79.3,  27 91.4 / 85.2,  54 145 / 132
  // The form that this rule takes is at most 5% slower than the other.
  const int cols = f8::token_cols(*p);
  const bool many = units > (cols == 16 ? 160 : cols == 32 ? 64 : 24) * (int64_t)sm_count;
  const size_t most = many ? f8::kMaxSmem : f8::kHalfSmem;
  p->many = many;
  for (p->up_stages = f8::kMaxStages; p->up_stages > 2 && f8::up_smem(*p) > most;) --p->up_stages;
  for (p->down_stages = f8::kMaxStages; p->down_stages > 2 && f8::down_smem(*p) > most;) --p->down_stages;
}

cudaError_t launch_fp8_moe(const MoeMaps& maps, const MoeParams& p, int sm_count, cudaStream_t stream) {
  const int col_tiles = (p.inner + f8::kUpCols - 1) / f8::kUpCols;
  const int grid = std::min(sm_count, p.active_max * col_tiles);
  return f8::with_token_cols(f8::token_cols(p), [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    CUtensorMap x = maps.x, g = maps.gate, u = maps.up, h = maps.h, d = maps.down;
    MoeParams q = p;
    void* up_args[] = {&x, &g, &u, &q};
    const cudaError_t e = f8::launch_pdl(reinterpret_cast<const void*>(f8::moe_up_kernel<NC>), grid, f8::up_smem(p), up_args,
                                         stream);
    if (e != cudaSuccess) return e;
    void* down_args[] = {&h, &d, &q};
    return f8::launch_pdl(reinterpret_cast<const void*>(f8::moe_down_kernel<NC>), p.down_grid, f8::down_smem(p), down_args,
                          stream);
  });
}

}  // namespace sgemm_impl
