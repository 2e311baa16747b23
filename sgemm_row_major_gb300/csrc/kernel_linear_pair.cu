// kernel_linear_pair.cu -- products of BF16 matrices on CTA pairs for sm_103a, with what a layer does to the sums.
//
//     linear:        Y = act(X W^T + bias) + R          gated:  H = act(X G^T) * (X U^T)
//     gradients:     D = A0 B0 (+ A1 B1)
//
// Up to three such products (jobs) run in one launch, their tiles one behind the other: a backward pass's products together
// fill the rounds of tiles better than each alone.  Where tiles are few and K is long, the K tiles of a tile are shared by
// several units, whose FP32 sums kernel_linear_join.cu adds.
//
// Clusters of two CTAs on one TPC compute 256 x TN tiles (TN 64, 128 or 256) with tcgen05.mma.cta_group::2.kind::f16,
// M = 256, N = TN, K = 16, both operands from shared memory: each CTA holds 128 rows of A and half of the tile's columns of
// B.  A gated tile has TN / 2 columns of each product: the even CTA's half of B is gate's rows, the odd one's up's, so every
// thread that reads the accumulator finds both products of an element in its own lane.  The epilogue runs over an accumulator
// 64 columns at a time while the next tile's products fill the other one.  The tensor cores' own accumulation is not
// round-to-nearest and drifts by about 1.5e-8 of the sum per instruction of 16 k (where signs are random; up to 1e-7 where the terms
// have one).  Where FP32 values leave the kernel (an FP32
// output, the scales of 8-bit values) only `fold` K tiles are summed in one accumulator, and these sums in FP32 registers;
// BF16 outputs take sums of up to 256 K tiles whole from the tensor memory (off by 1.6e-5 of the sum at that length where the terms'
// signs are random and by 7.5e-5 where they have one sign; their own rounding is 2e-3), which leaves the next tile's products a whole
// tile's time to overlap with the epilogue; longer ones are folded in parts of that many.
//
// Either operand may be stored along K or across it: the tensor core reads both orders, so a gradient's product takes the
// weights and activations as the forward pass left them.
//
// Warp 0 loads (TMA, 5 stages of 32 KB or 8 of 24), warp 1 of the even CTA issues the products, warps 4-11 fold and write.  Persistent
// clusters take tiles round robin in an order that keeps 8 rows of tiles together (their A and B panels stay in L2).
//
// Large calls are bound by the tensor cores: 82 to 88 % busy (4096 tokens, 4096 -> 8192, 8-bit values kept: gated 303 us, one
// product 159; a gated block's three gradients 618), and by the power limit in runs of many.  On the GPU 8192 x 4096 -> 8192 gated
// takes 604 us, 1.82 PFLOP/s.
#include "linear_common.cuh"

namespace sgemm_impl {
namespace lin {
namespace {

using namespace tc;

constexpr int BM = 256, BMC = 128, BK = 64;
constexpr int kPart = 128 * BK * 2;       // 16 KB: A's tile in one CTA
constexpr int kFirstFold = 4;             // warps 0 and 1: loads, products
constexpr int kFoldWarps = 8;
constexpr int kThreads = 32 * (kFirstFold + kFoldWarps);
static_assert(kThreads == kLinearPairThreads, "the plan's figure");
// 384 threads are launched with 168 registers each; the four warps that move data give most of theirs to the folders:
// 128 x 40 + 256 x 232 = 384 x 168.
constexpr int kMoverRegs = 40, kFoldRegs = 232;
static_assert(128 * kMoverRegs + 32 * kFoldWarps * kFoldRegs <= kThreads * 168, "registers at launch");
constexpr int kMaxBufs = 4;
constexpr uint32_t kTmemCols = 512;

// Shared memory by the tile's width: narrow tiles take less of it per K tile and as long to arrive, so they get more stages.
template <int TN>
struct Ring {
  static constexpr int kPartB = TN == 256 ? kPart : kPart / 2;  // (64 columns across K are copied as a block of 64)
  static constexpr int kStageBytes = kPart + kPartB;
  static constexpr int kStages = TN == 256 ? 5 : 8;
  static constexpr int kOutBytes = TN == 256 ? 8 * 1024 : 4 * 1024;  // per folding warp: pieces of 2 KB (BF16) or 4 KB (FP32)
  static constexpr int kSmem = kStages * kStageBytes + kFoldWarps * kOutBytes + 1024;
  static_assert(kSmem + 1536 <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int32_t inner, int32_t outer) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(inner), "r"(outer), "r"(0)
      : "memory");
}

template <int N>
__device__ __forceinline__ void add_to(float* v, const float* x) {
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    const float2 s = add(make_float2(v[k], v[k + 1]), make_float2(x[k], x[k + 1]));
    v[k] = s.x;
    v[k + 1] = s.y;
  }
}

// A folding warp's pieces of an output, 32 rows each: written to shared memory in the output's type, in rows of 64 (32 columns of
// BF16) or 128 bytes (64 of BF16, 32 of FP32) with the swizzle of that width, then by TMA
// or by the lanes.  Rows of 128 bytes halve what the copy engine has to do for a tile.
template <int BYTES>
struct Pieces {
  uint8_t* buf;
  int at;     // the next piece's place
  bool wide;  // places of 4 KB, else of 2 KB
  __device__ __forceinline__ void set(bool w) {
    if (w == wide) return;
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    wide = w;
    at = 0;
  }
  __device__ __forceinline__ uint8_t* next() {
    constexpr int kNarrow = BYTES / 2048, kWide = BYTES / 4096;
    uint8_t* p = buf + at * (wide ? 4096 : 2048);
    at = (at + 1) & (wide ? kWide - 1 : kNarrow - 1);
    // the copy that read this place before is done reading
    if ((threadIdx.x & 31) == 0) {
      if (wide) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kWide - 1) : "memory");
      else      asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kNarrow - 1) : "memory");
    }
    __syncwarp();
    return p;
  }
  // Sends a piece off (a group without a copy where it lies outside: places and groups advance together).
  __device__ __forceinline__ void copy(const uint8_t* p, const CUtensorMap* map, bool inside, int row0, int col0) {
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0 && inside)
      asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                   "r"(smem_addr(p)), "r"(col0), "r"(row0), "r"(0)
                   : "memory");
    commit();
  }
  __device__ __forceinline__ void commit() {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
};

// W columns (32 or 64) of this lane's row of D (or of what is kept) go out.  TMA writes whole 16 bytes of a row; what is left of
// it, and everything where rows are not aligned (tma: 0), is written by lanes that run along the rows.
template <bool F32, int W, int BYTES>
__device__ __forceinline__ void emit(Pieces<BYTES>& pieces, const CUtensorMap* map, bool tma, void* base, int64_t ld, const LinearOut& o,
                                     const LinearJob& j, unsigned site, int row0, int col0, const float (&v)[W]) {
  using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
  constexpr int kCols = F32 ? 32 : W, kBytes = kCols * (int)sizeof(T);  // of a piece's row
  const int lane = threadIdx.x & 31;
  const int by_tma = tma ? j.N & ~(16 / (int)sizeof(T) - 1) : 0;
#pragma unroll
  for (int h = 0; h < W / kCols; ++h) {
    uint8_t* at = pieces.next();
    const int first = col0 + kCols * h;
    // 16-byte unit e of row r
    const auto unit = [&](int r, int e) { return at + r * kBytes + 16 * (e ^ (kBytes == 128 ? r & 7 : (r >> 1) & 3)); };
#pragma unroll
    for (int e = 0; e < kBytes / 16; ++e) {
      const float* x = v + kCols * h + 16 / (int)sizeof(T) * e;
      if constexpr (F32)
        *reinterpret_cast<float4*>(unit(lane, e)) = make_float4(x[0], x[1], x[2], x[3]);
      else
        *reinterpret_cast<uint4*>(unit(lane, e)) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    }
    if (tma) pieces.copy(at, map, row0 < j.M && first < by_tma, row0, first);
    else     __syncwarp();
    if (first + kCols > by_tma && by_tma < j.N && row0 < j.M) {
      const int rows = min(32, j.M - row0);
#pragma unroll 1
      for (int c = max(first, by_tma) + lane; c < min(first + kCols, j.N); c += 32) {
        if (!in_range(o.guard.fault, o.guard.word, site, (int64_t)row0 * ld + c, (rows - 1) * ld + 1, extent(j.M, ld, j.N))) continue;
        T* d = static_cast<T*>(base) + (int64_t)row0 * ld + c;
        const int byte = (c - first) * (int)sizeof(T);
#pragma unroll 8
        for (int r = 0; r < rows; ++r, d += ld) *d = *reinterpret_cast<const T*>(unit(r, byte >> 4) + (byte & 15));
      }
      __syncwarp();
    }
    if (!tma) pieces.commit();
  }
}

// W values of the bias, or of one row of the residual (whose rows are aligned), sent for before the sums are waited for: 8 at a
// time where they are aligned (vec), at a row's end and otherwise one by one.
template <int W>
struct Ahead {
  uint4 c[W / 8];
  // p: the first of them, of which `left` are there, at element `at` of the `size` of its buffer
  __device__ __forceinline__ void load(const Guard& g, const __nv_bfloat16* p, bool vec, int left, int64_t at, int64_t size) {
#pragma unroll
    for (int e = 0; e < W / 8; ++e) {
      const int n = min(8, left - 8 * e);
      c[e] = make_uint4(0u, 0u, 0u, 0u);
      if (n <= 0 || !in_range(g.fault, g.word, f8::kSiteIn, at + 8 * e, n, size)) continue;
      if (vec && n == 8) {
        c[e] = reinterpret_cast<const uint4*>(p)[e];
      } else {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < n) w[k / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[8 * e + k] << (16 * (k % 2));
        c[e] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  __device__ __forceinline__ void add(float (&v)[W]) const {
#pragma unroll
    for (int e = 0; e < W / 8; ++e) {
      Chunk<__nv_bfloat16> b;
      float x[8];
      b.raw = c[e];
      b.get(x);
      add_to<8>(&v[8 * e], x);
    }
  }
  __device__ __forceinline__ void bias(const LinearOut& o, const LinearJob& j, int col0) {
    load(o.guard, static_cast<const __nv_bfloat16*>(o.bias) + col0, o.bias_vec, j.N - col0, col0, j.N);
  }
  __device__ __forceinline__ void residual(const LinearOut& o, const LinearJob& j, int row, int col0) {
    const int64_t at = (int64_t)row * o.ldr + col0;
    load(o.guard, static_cast<const __nv_bfloat16*>(o.residual) + at, true, row < j.M ? j.N - col0 : 0, at, extent(j.M, o.ldr, j.N));
  }
};

// Asks for `cols` values of the residual in one row to be brought to L2, while the tile's products run.
__device__ __forceinline__ void prefetch_residual(const LinearOut& o, const LinearJob& j, int row, int col0, int cols) {
  const int n = min(cols, j.N - col0);
  if (row >= j.M || n <= 0 || !r_ok(o, j, row, col0, n)) return;
  const char* p = reinterpret_cast<const char*>(static_cast<const __nv_bfloat16*>(o.residual) + (int64_t)row * o.ldr + col0);
  for (int at = 0; at < 2 * n; at += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + at));
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 2 * n - 2));
}

// 32 codes of one row.  CHECK: some value may be infinite.
template <bool CHECK>
__device__ __forceinline__ void put_codes(const LinearOut& o, const LinearJob& j, int which, int row, int col0, const float* v, float inv) {
  const LinearKept& k = o.kept[which];
  uint32_t u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 a = mul(make_float2(v[4 * e], v[4 * e + 1]), both(inv)), b = mul(make_float2(v[4 * e + 2], v[4 * e + 3]), both(inv));
    u[e] = f8::codes2<CHECK>(a.x, a.y, false) | (f8::codes2<CHECK>(b.x, b.y, false) << 16);
  }
  if (row >= j.M || col0 >= j.N) return;
  const int n = min(32, j.N - col0);
  if (!kept_ok(o, j, which, row, col0, n)) return;
  uint8_t* d = static_cast<uint8_t*>(k.data) + (int64_t)row * k.ld + col0;
  if (k.vec && n == 32) {
    reinterpret_cast<uint4*>(d)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    reinterpret_cast<uint4*>(d)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (e < n) d[e] = (uint8_t)(u[e / 4] >> (8 * (e % 4)));
  }
}

// The largest finite |v| so far (a NaN is never the larger one; infinities are looked for only where there are some, and
// remembered).
template <int W>
__device__ __forceinline__ float largest_of(float m, bool& infinite, const float (&v)[W]) {
  float x = 0.0f, y = 0.0f;
#pragma unroll
  for (int k = 0; k < W; k += 2) {
    x = fmaxf(x, fabsf(v[k]));
    y = fmaxf(y, fabsf(v[k + 1]));
  }
  x = fmaxf(x, y);
  if (x > f8::kMaxFloat) {
    infinite = true;
    x = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) x = fmaxf(x, f8::finite_abs(v[k]));
  }
  return fmaxf(m, x);
}

// W columns of this thread's TMEM lane.
template <int W>
__device__ __forceinline__ void tmem_get(uint32_t taddr, float (&v)[W]) {
#pragma unroll
  for (int h = 0; h < W; h += 32) tmem_ld32(taddr + (uint32_t)h, v + h);
}
template <int W>
__device__ __forceinline__ void tmem_put(uint32_t taddr, const float (&v)[W]) {
#pragma unroll
  for (int h = 0; h < W; h += 16) tmem_st16(taddr + (uint32_t)h, *reinterpret_cast<const float(*)[16]>(&v[h]));
}

// The job of a unit of work, the tile and the K tiles [g0, g1) (over both segments) it takes.  SHARED: some job's tiles are
// several units.
template <bool SHARED>
struct Place {
  int job, tm, tn, slice, g0, g1;
  __device__ __forceinline__ static int units(const LinearJob& j) { return j.tiles_m * j.tiles_n * (SHARED ? j.split : 1); }
  __device__ __forceinline__ Place(const LinearPairParams& p, int unit) : job(0), slice(0), g0(0) {
    // (written out: with a call of units() the 256-wide folding kernel spilled 176 bytes, so it spills 20)
    if (SHARED) {
      while (unit >= units(p.job[job])) unit -= units(p.job[job]), ++job;
    } else {
      while (unit >= p.job[job].tiles_m * p.job[job].tiles_n) unit -= p.job[job].tiles_m * p.job[job].tiles_n, ++job;
    }
    const LinearJob& j = p.job[job];
    g1 = j.k_tiles * j.segments;
    if (SHARED && j.split > 1) {  // the units of a tile one behind the other
      slice = unit % j.split;
      unit /= j.split;
      g0 = (int)((int64_t)g1 * slice / j.split);
      g1 = (int)((int64_t)g1 * (slice + 1) / j.split);
    }
    tile_coords(unit, j.tiles_m, j.tiles_n, tm, tn);
  }
};

// TN: the accumulator's columns.  GATED: half of them are gate's, half up's.  FOLD: FP32 values leave the kernel (an FP32
// output, scales of 8-bit values) or a sum is long, so a job may add several accumulators in registers; without that the epilogue has room for
// 64 columns at a time everywhere.  SHARED: some job's K is shared by several units; sums are written and nothing else is done.
// (A form of its own: with the sharing in all of them 16384 tokens, 256 -> 2048 gated, kept in 8 bits, took 59.4 us, not 56.3.)
template <int TN, bool GATED, bool FOLD, bool SHARED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearPairParams p) {
  extern __shared__ uint8_t smem_raw[];
  using R = Ring<TN>;
  constexpr int kStages = R::kStages, kStageBytes = R::kStageBytes;
  constexpr int halfn = TN / 2;   // columns of B this CTA loads
  constexpr int TD = GATED ? TN / 2 : TN;  // the tile's columns of D
  constexpr int bufs = (int)kTmemCols / TN < kMaxBufs ? (int)kTmemCols / TN : kMaxBufs;
  __shared__ __align__(8) uint64_t full[kStages], done[kStages];
  __shared__ __align__(8) uint64_t acc_full[bufs], acc_empty[bufs];
  // a group of 128 columns held by two warps: the second one's largest values, and then both's
  __shared__ __align__(8) uint64_t max_asked[4], max_told[4];
  __shared__ float largest[GATED ? 2 : 1][BMC];
  __shared__ __align__(8) uint64_t fin;
  __shared__ uint32_t tmem_slot;

  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  const uint32_t sbase = raw_addr + pad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cl = (int)cluster_id_x();
  int tiles = 0;
  for (int n = 0; n < p.jobs; ++n) tiles += Place<SHARED>::units(p.job[n]);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&done[s]), 1);
    }
    for (int b = 0; b < bufs; ++b) {
      mbar_init(smem_addr(&acc_full[b]), 1);
      mbar_init(smem_addr(&acc_empty[b]), 2 * kFoldWarps);
    }
    for (int q = 0; q < 4; ++q) {
      mbar_init(smem_addr(&max_asked[q]), 1);
      mbar_init(smem_addr(&max_told[q]), 1);
    }
    mbar_init(smem_addr(&fin), 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_addr(&tmem_slot), kTmemCols);
  tmem_fence_before_sync();
  cluster_sync();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  // (not before this CTA has its tensor memory: a dependent that took it first would wait for this grid, and this grid for it)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // launched as a programmatic dependent: what the stream's kernel before this one wrote is read, and what it read is
  // written, only from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp < kFirstFold) {
    f8::fewer_registers<kMoverRegs>();
    if (warp == 0) {
      // ------------------------------------------------ loads (each CTA: its rows of A, its columns of B)
      if (lane == 0) {
        prefetch_tensormap(&maps.op[p.job[0].a[0]]);
        prefetch_tensormap(&maps.op[p.job[0].b[GATED ? rank : 0]]);
      }
      __syncwarp();
      const uint32_t full0 = map_to_rank(smem_addr(&full[0]), 0);
      int t = 0, s = 0;
      uint32_t lap = 0;
      bool ok = true;
      for (int tile = cl; ok && tile < tiles; tile += p.clusters) {
        const Place<SHARED> at(p, tile);
        const LinearJob& j = p.job[at.job];
        const uint32_t bytes = 2u * (part_bytes(j.a_mn, BMC) + part_bytes(j.b_mn, halfn));  // both CTAs'
        const int m0 = at.tm * BM + BMC * (int)rank, n0 = GATED ? at.tn * TD : at.tn * TN + halfn * (int)rank;
        const int a_mn = j.a_mn, b_mn = j.b_mn, kt = j.k_tiles;
        for (int segment = 0; ok && segment < j.segments; ++segment) {
          const CUtensorMap *ma = &maps.op[j.a[segment]], *mb = &maps.op[j.b[GATED ? (int)rank : segment]];
          const int end = SHARED ? min(kt, at.g1 - segment * kt) : kt;
          for (int k = SHARED ? max(0, at.g0 - segment * kt) : 0; k < end; ++k, ++t) {
            if (lap > 0 && !poll_wait(smem_addr(&done[s]), (lap - 1) & 1u, p.timeout_ns)) {
              if (lane == 0) atomicOr(p.fault, (unsigned)kFaultEmptyWait);
              ok = false;
              break;
            }
            if (elect_one()) {
              // both CTAs' loads complete on the even CTA's barrier, which expects all their bytes
              const uint32_t fb = full0 + 8u * (uint32_t)s;
              if (rank == 0) mbar_arrive_expect_tx(smem_addr(&full[s]), bytes);
              const uint32_t a = sbase + (uint32_t)(s * kStageBytes);
              const auto load = [&](uint32_t dst, const CUtensorMap* map, int inner, int outer) { tma_load_pair(dst, map, fb, inner, outer); };
              load_part(load, a, ma, a_mn, m0, k * BK, BMC);
              load_part(load, a + kPart, mb, b_mn, n0, k * BK, halfn);
            }
            if (++s == kStages) {
              s = 0;
              ++lap;
            }
          }
        }
      }
      // leave only when every copy into shared memory has landed (the odd CTA's warp 1 waits for the products that read its
      // last stages)
      if (rank == 0)
        for (int u = t > kStages ? t - kStages : 0; u < t; ++u)
          if (!poll_wait(smem_addr(&full[u % kStages]), (uint32_t)(u / kStages) & 1u, p.timeout_ns) && lane == 0)
            atomicOr(p.fault, (unsigned)kFaultDrainWait);
    } else if (warp == 1) {
      int t = 0;  // K tiles whose products have been issued (odd CTA: will be)
      if (rank != 0) {
        for (int tile = cl; tile < tiles; tile += p.clusters) {
          const Place<SHARED> at(p, tile);
          t += at.g1 - at.g0;
        }
      } else {
        // ---------------------------------------------- products (even CTA)
        const uint32_t desc0 = desc_lo(sbase);
        int s = 0, b = 0;
        uint32_t s_lap = 0, b_lap = 0;
        bool ok = true;
        for (int tile = cl; ok && tile < tiles; tile += p.clusters) {
          const Place<SHARED> at(p, tile);
          const LinearJob& j = p.job[at.job];
          const uint32_t astep = step_of(j.a_mn), bstep = step_of(j.b_mn), idesc = j.idesc;
          const int kt = at.g1 - at.g0;
          int n = j.fold0;  // a chunk: the K tiles of one accumulator
          for (int g = 0; ok && g < kt; g += n, n = j.fold) {
            n = min(n, kt - g);
            ok = b_lap == 0 || poll_wait(smem_addr(&acc_empty[b]), (b_lap - 1) & 1u, p.timeout_ns);
            tmem_fence_after_sync();
            for (int i = 0; ok && i < n; ++i) {
              ok = poll_wait(smem_addr(&full[s]), s_lap & 1u, p.timeout_ns);
              if (!ok) break;
              tmem_fence_after_sync();
              if (elect_one()) {
                const uint32_t acc = tmem + (uint32_t)(b * TN);
                const uint32_t ad = desc0 + (uint32_t)(s * (kStageBytes >> 4)), bd = ad + (kPart >> 4);
#pragma unroll
                for (uint32_t ks = 0; ks < BK / 16; ++ks)
                  mma_bf16_pair(acc, make_desc(ad + ks * astep), make_desc(bd + ks * bstep), idesc, i == 0 && ks == 0 ? 0u : 1u);
                mma_commit_pair(smem_addr(&done[s]));  // in both CTAs: stage s is free
                if (i == n - 1) mma_commit_pair(smem_addr(&acc_full[b]));
              }
              __syncwarp();
              ++t;
              if (++s == kStages) {
                s = 0;
                ++s_lap;
              }
            }
            if (++b == bufs) {
              b = 0;
              ++b_lap;
            }
          }
        }
        if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
      }
      // leave only when every product has completed and its commits have landed in this CTA
      for (int u = t > kStages ? t - kStages : 0; u < t; ++u)
        if (!poll_wait(smem_addr(&done[u % kStages]), (uint32_t)(u / kStages) & 1u, p.timeout_ns)) {
          if (lane == 0) atomicOr(p.fault, (unsigned)kFaultDrainWait);
          break;
        }
    }
  } else {
    f8::more_registers<kFoldRegs>();
    // ------------------------------------------------ folders, then the epilogue (both CTAs)
    const LinearOut& o = p.out;
    const int q = warp & 3;                     // TMEM lane quarter this warp may access
    const int part = (warp - kFirstFold) >> 2;  // which half of the tile's columns
    constexpr int cols = TD / 2;                // of D, per thread
    constexpr int loads = TN / 64;              // 32 accumulator columns at a time
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(cols * part);
    // the accumulator column of load e: gated, the first half of the loads are gate's columns, the others up's
    const auto column = [](int e) { return GATED && e >= loads / 2 ? TN / 2 + 32 * (e - loads / 2) : 32 * e; };
    Pieces<R::kOutBytes> pieces{smem_raw + pad + kStages * kStageBytes + (warp - kFirstFold) * R::kOutBytes, 0, false};
    bool ok = true;
    int b = 0;
    uint32_t b_lap = 0, asked = 0;  // tiles whose largest values have been exchanged
    const auto fetch = [&](int tile) {  // has a tile's residual brought to L2
      if (GATED || SHARED || !o.residual || tile >= tiles) return;
      const Place<SHARED> to(p, tile);
      prefetch_residual(o, p.job[to.job], to.tm * BM + BMC * (int)rank + 32 * q + lane, to.tn * TD + cols * part, cols);
    };
    fetch(cl);
    fetch(cl + p.clusters);
    for (int tile = cl; ok && tile < tiles; tile += p.clusters) {
      const Place<SHARED> at(p, tile);
      const LinearJob& j = p.job[at.job];
      const int row0 = (SHARED ? at.slice * j.rows_apart : 0) + at.tm * BM + BMC * (int)rank + 32 * q, row = row0 + lane;
      const int c0 = at.tn * TD + cols * part;  // this thread's first column of D
      const int kt = at.g1 - at.g0;
      uint32_t acc;
      const auto next = [&] {  // waits for the next accumulator
        ok = poll_wait(smem_addr(&acc_full[b]), b_lap & 1u, p.timeout_ns);
        if (!ok && lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
        tmem_fence_after_sync();
        acc = tq + (uint32_t)(b * TN);
        return ok;
      };
      const auto release = [&] {  // the accumulator has been read: hand it back to the issuer
        tmem_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(smem_addr(&acc_empty[b]), 0);
        if (++b == bufs) {
          b = 0;
          ++b_lap;
        }
      };
      bool several = false;
      if constexpr (FOLD) {
        several = kt > j.fold0;
        if (several) {
          // several accumulators: all but the last are added in registers, and these sums to the last one where it lies
          float sum[TN / 2];
#pragma unroll
          for (int e = 0; e < TN / 2; ++e) sum[e] = 0.0f;
          for (int g = j.fold0; g < kt; g += j.fold) {  // (g: K tiles up to this accumulator's end)
            if (!next()) break;
#pragma unroll
            for (int e = 0; e < 2 * loads; ++e) {
              float v[16];
              tmem_ld16(acc + (uint32_t)(column(e / 2) + 16 * (e % 2)), v);
              tmem_wait_ld();
              if (e == 2 * loads - 1) release();
              tmem_ld_ready(v);
              add_to<16>(&sum[16 * e], v);
            }
          }
          if (!ok || !next()) break;
#pragma unroll
          for (int e = 0; e < 2 * loads; ++e) {
            const uint32_t at16 = acc + (uint32_t)(column(e / 2) + 16 * (e % 2));
            float v[16];
            tmem_ld16(at16, v);
            tmem_wait_ld();
            tmem_ld_ready(v);
            add_to<16>(v, &sum[16 * e]);
            tmem_st16(at16, v);
          }
          tmem_wait_st();
        }
      }
      if (!several && !next()) break;
      // ---------------------------------------------- epilogue, W columns at a time
      constexpr int W = linear_pair_box(TN, GATED, FOLD);
      constexpr uint32_t up = TN / 2;  // gated: from a column of gate to up's
      pieces.set(W == 64 || (FOLD && j.f32 != 0));
      const CUtensorMap* map_d = &maps.d[at.job];
      float inv[2] = {1.0f, 1.0f};       // of the scales of what is kept in 8 bits
      bool odd = false;                  // an infinity among them
      bool add_bias = !GATED && !SHARED && o.bias;  // still to be done
      if (!SHARED && o.keep) {
        // what is kept in BF16, or the largest values of what is kept in 8 bits; the bias is added where the sums lie
        float m[2] = {0.0f, 0.0f};
#pragma unroll 1
        for (int c = 0; c < cols; c += W) {
          float v[W];
          Ahead<W> bias;
          tmem_get(acc + (uint32_t)c, v);
          if (add_bias) bias.bias(o, j, c0 + c);
          tmem_wait_ld();
          tmem_ld_ready(v);
          if (add_bias) {
            bias.add(v);
            tmem_put(acc + (uint32_t)c, v);
          }
          if (!FOLD || o.keep == 1) emit<false>(pieces, &maps.kept[0], o.kept[0].vec, o.kept[0].data, o.kept[0].ld, o, j, f8::kSiteCodes, row0, c0 + c, v);
          else                      m[0] = largest_of(m[0], odd, v);
          if constexpr (GATED) {
            tmem_get(acc + up + (uint32_t)c, v);
            tmem_wait_ld();
            tmem_ld_ready(v);
            if (!FOLD || o.keep == 1) emit<false>(pieces, &maps.kept[1], o.kept[1].vec, o.kept[1].data, o.kept[1].ld, o, j, f8::kSiteCodes, row0, c0 + c, v);
            else                      m[1] = largest_of(m[1], odd, v);
          }
        }
        if (add_bias) tmem_wait_st();
        add_bias = false;
        if (FOLD && o.keep == 2) {
          odd = __any_sync(0xffffffffu, odd);
          if (cols < 128) {  // the other half of the group is with the warp of the other column half
            float* slot = &largest[0][32 * q + lane];
            constexpr int kUp = GATED ? BMC : 0;
            if (part == 1) {
              slot[0] = m[0];
              if (GATED) slot[kUp] = m[1];
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&max_asked[q]));
            }
            ok = poll_wait(smem_addr(part == 1 ? &max_told[q] : &max_asked[q]), asked & 1u, p.timeout_ns);
            ++asked;
            if (!ok) {
              if (lane == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
              break;
            }
            m[0] = fmaxf(m[0], slot[0]);
            if (GATED) m[1] = fmaxf(m[1], slot[kUp]);
            if (part == 0) {
              slot[0] = m[0];
              if (GATED) slot[kUp] = m[1];
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&max_told[q]));
            }
          }
#pragma unroll
          for (int w = 0; w < (GATED ? 2 : 1); ++w) {
            const float scale = f8::group_scale(m[w], kMaxE4M3);
            if (row < j.M && c0 < j.N && c0 % 128 == 0) put_scale(o, j, w, row, c0 >> 7, scale);
            inv[w] = __fdiv_rn(1.0f, scale);
          }
        }
      }
#pragma unroll 1
      for (int c = 0; c < cols; c += W) {
        const bool last = c + W == cols;
        const auto codes = [&](int which, const float (&x)[W]) {
#pragma unroll
          for (int h = 0; h < W; h += 32) {
            if (odd) put_codes<true>(o, j, which, row, c0 + c + h, x + h, inv[which]);
            else     put_codes<false>(o, j, which, row, c0 + c + h, x + h, inv[which]);
          }
        };
        float v[W];
        tmem_get(acc + (uint32_t)c, v);
        if constexpr (GATED) {
          float u[W];
          tmem_get(acc + up + (uint32_t)c, u);
          tmem_wait_ld();
          if (last) release();
          tmem_ld_ready(v);
          tmem_ld_ready(u);
          if (FOLD && o.keep == 2) {
            codes(0, v);
            codes(1, u);
          }
          with_act(o.act, [&](auto act) {
#pragma unroll
            for (int k = 0; k < W; k += 2) {
              const float2 h = mul(act_of<decltype(act)::value>(make_float2(v[k], v[k + 1])), make_float2(u[k], u[k + 1]));
              v[k] = h.x;
              v[k + 1] = h.y;
            }
          });
          emit<false>(pieces, map_d, j.d_tma, j.d, j.ldd, o, j, f8::kSiteOut, row0, c0 + c, v);
        } else {
          Ahead<W> residual, bias;
          if (!SHARED && o.residual) residual.residual(o, j, row, c0 + c);
          if (add_bias) bias.bias(o, j, c0 + c);
          tmem_wait_ld();
          if (last) release();
          tmem_ld_ready(v);
          if (add_bias) bias.add(v);
          if (FOLD && !SHARED && o.keep == 2) codes(0, v);
          if (!SHARED) with_act(o.act, [&](auto act) {
#pragma unroll
            for (int k = 0; k < W; k += 2) {
              const float2 f = act_of<decltype(act)::value>(make_float2(v[k], v[k + 1]));
              v[k] = f.x;
              v[k + 1] = f.y;
            }
          });
          if (!SHARED && o.residual) residual.add(v);
          if (FOLD && j.f32) emit<true>(pieces, map_d, j.d_tma, j.d, j.ldd, o, j, f8::kSiteOut, row0, c0 + c, v);
          else               emit<false>(pieces, map_d, j.d_tma, j.d, j.ldd, o, j, f8::kSiteOut, row0, c0 + c, v);
        }
      }
      fetch(tile + 2 * p.clusters);  // (its place need not be held during the sums here)
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  tmem_fence_before_sync();
  __syncthreads();
  // Bounded handshake of the two CTAs: neither releases its TMEM or exits while the other may still arrive on its barriers
  // or have products read its shared memory and TMEM.
  if (threadIdx.x == 0) {
    mbar_arrive_remote(smem_addr(&fin), rank ^ 1u);
    if (!mbar_wait(smem_addr(&fin), 0u, p.timeout_ns)) atomicOr(p.fault, (unsigned)kFaultDrainWait);
  }
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// f(kernel) for a tile width and form.
template <bool FOLD, bool SHARED, typename F>
cudaError_t with_form(int tile_n, bool gated, const F& f) {
  constexpr bool kGated = !SHARED;  // (K of gated products is not shared)
  if (gated && (tile_n == 64 || SHARED)) return cudaErrorInvalidValue;
  switch (tile_n) {
    case 256: return gated ? f(linear_pair_kernel<256, kGated, FOLD, SHARED>) : f(linear_pair_kernel<256, false, FOLD, SHARED>);
    case 128: return gated ? f(linear_pair_kernel<128, kGated, FOLD && SHARED, SHARED>) : f(linear_pair_kernel<128, false, FOLD, SHARED>);  // (gated: whole sums for BF16 alone)
    case 64: return f(linear_pair_kernel<64, false, FOLD, SHARED>);
    default: return cudaErrorInvalidValue;
  }
}
template <typename F>
cudaError_t with_kernel(int tile_n, bool gated, LinearPairForm form, const F& f) {
  switch (form) {
    case LinearPairForm::kWhole: return with_form<false, false>(tile_n, gated, f);
    case LinearPairForm::kFold: return with_form<true, false>(tile_n, gated, f);
    default: return with_form<true, true>(tile_n, gated, f);
  }
}

}  // namespace
}  // namespace lin

int linear_pair_stages(int tile_n) { return tile_n == 256 ? lin::Ring<256>::kStages : lin::Ring<128>::kStages; }
int64_t linear_pair_smem(int tile_n) { return tile_n == 256 ? lin::Ring<256>::kSmem : lin::Ring<128>::kSmem; }

cudaError_t prepare_linear_pair() {
  for (int tile_n : kLinearPairTiles)
    for (int n = 0; n < 6; ++n) {
      const bool gated = n >= 3;
      const LinearPairForm form = (LinearPairForm)(n % 3);
      if (gated && (tile_n == 64 || form == LinearPairForm::kShared)) continue;
      const cudaError_t e = lin::with_kernel(tile_n, gated, form, [&](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)linear_pair_smem(tile_n));
      });
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

cudaError_t launch_linear_pair(int tile_n, bool gated, LinearPairForm form, const LinearMaps& maps, const LinearPairParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)p.clusters);
  cfg.blockDim = dim3(lin::kThreads);
  cfg.dynamicSmemBytes = (size_t)linear_pair_smem(tile_n);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return lin::with_kernel(tile_n, gated, form, [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, maps, p); });
}

}  // namespace sgemm_impl
