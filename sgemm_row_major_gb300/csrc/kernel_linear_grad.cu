// kernel_linear_grad.cu -- the elementwise part of the backward passes of a layer and of a gated block, for sm_103a, and the
// aligned BF16 copies of operands that the tensor cores' loads cannot read as they are.
//
//     layer:  dA = dY * act'(A),  dbias = sum over the rows of dA
//     gated:  dA = dH * B * act'(A),  dB = dH * act(A),  H = act(A) * B
//
// A and B as the forward pass kept them: BF16, or 8-bit codes times the scale of their group of 128.  One pass over the data,
// bound by the memory and nearly as much by the instructions of an activation's derivative (two values at a time in packed
// arithmetic).  A thread takes 8 columns of a row (16 bytes of BF16, 8 of codes); what it
// reads of its next four rows is on its way to shared memory while it works on one (in registers the loads of two rows covered
// half of the memory's latency).  Column sums are held per thread in FP32 and joined within the CTA, then
// by a cluster of up to 8 CTAs that share the rows of a strip, or (many rows, where the clusters' CTAs are too few to fill the
// chip, and wide strips) by a second kernel; always in a fixed order.
// Gated, 4096 x 8192 values kept in BF16, with H: 58 us, 6.1 TB/s.
#include <algorithm>

#include "linear_common.cuh"

namespace sgemm_impl {
namespace lin {
namespace {

constexpr int kThreads = 256, kWide = 256, kNarrow = 64;  // columns of a strip
constexpr int kStages = 4;        // rows ahead per thread
constexpr int kBatch = 2;         // without alignment: rows whose loads are on their way together
constexpr int kExpandChunks = 4;  // the same of the copies, in chunks of 8 columns

// 8 consecutive values of codes and their scale.
__device__ __forceinline__ void decode(uint2 c, float scale, float2 (&x)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((e < 2 ? c.x : c.y) >> (16 * (e % 2))), __NV_E4M3);
    x[e] = mul(__half22float2(__half2(h)), both(scale));
  }
}

// 8 consecutive values at any alignment, n of them there, sent for and then waited for.
template <bool CODES>
struct KeptLoad;
template <>
struct KeptLoad<false> {
  f8::Loading<__nv_bfloat16, false> v;
  __device__ __forceinline__ void load(const LinearKeptIn& k, int64_t rows, int cols, int64_t row, int col, int n, const Guard& g) {
    const f8::Rows<__nv_bfloat16> m(k.data, rows, k.ld, cols, g);
    v.load(m.base + row * k.ld + col, n, m);
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const { v.get().get(&x[0].x); }
};
template <>
struct KeptLoad<true> {
  uint2 c;
  float s;
  __device__ __forceinline__ void load(const LinearKeptIn& k, int64_t rows, int cols, int64_t row, int col, int n, const Guard& g) {
    c = make_uint2(0u, 0u);
    s = 0.0f;
    if (n <= 0) return;
    const uint8_t* base = static_cast<const uint8_t*>(k.data);
    const int64_t at = row * k.ld + col;
    if (!in_range(g.fault, g.word, f8::kSiteCodes, at, n, extent(rows, k.ld, cols))) return;
    s = get_at(g, f8::kSiteScale, k.scale, row * k.lds + (col >> 7), extent(rows, k.lds, (cols + 127) / 128));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) (e < 4 ? c.x : c.y) |= (uint32_t)base[at + e] << (8 * (e % 4));
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const { decode(c, s, x); }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
  else                       asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst)), "l"(src), "n"(BYTES) : "memory");
}

// 8 consecutive values that can be read at once, copied to shared memory ahead: a place per thread and stage, which no other
// thread reads.
template <bool CODES>
struct KeptRing;
template <>
struct KeptRing<false> {
  uint4 v[kStages][kThreads];
  __device__ __forceinline__ void copy(int s, const LinearKeptIn& k, int64_t rows, int cols, int64_t row, int col, const Guard& g) {
    const int64_t at = row * k.ld + col;
    if (in_range(g.fault, g.word, f8::kSiteIn, at, 8, extent(rows, k.ld, cols))) copy_async<16>(&v[s][threadIdx.x], static_cast<const __nv_bfloat16*>(k.data) + at);
  }
  __device__ __forceinline__ void get(int s, float2 (&x)[4]) const {
    Chunk<__nv_bfloat16> c;
    c.raw = v[s][threadIdx.x];
    c.get(&x[0].x);
  }
};
template <>
struct KeptRing<true> {
  uint2 c[kStages][kThreads];
  float scale[kStages][kThreads];
  __device__ __forceinline__ void copy(int s, const LinearKeptIn& k, int64_t rows, int cols, int64_t row, int col, const Guard& g) {
    const int64_t at = row * k.ld + col, group = row * k.lds + (col >> 7);
    if (in_range(g.fault, g.word, f8::kSiteCodes, at, 8, extent(rows, k.ld, cols))) copy_async<8>(&c[s][threadIdx.x], static_cast<const uint8_t*>(k.data) + at);
    if (in_range(g.fault, g.word, f8::kSiteScale, group, 1, extent(rows, k.lds, (cols + 127) / 128))) copy_async<4>(&scale[s][threadIdx.x], k.scale + group);
  }
  __device__ __forceinline__ void get(int s, float2 (&x)[4]) const { decode(c[s][threadIdx.x], scale[s][threadIdx.x], x); }
};

// 8 values as BF16, n of them there, to a row of an aligned (VEC) or any other matrix.
template <bool VEC>
__device__ __forceinline__ void put8(void* base, int64_t ld, int64_t rows, int cols, int64_t row, int col, int n, const float2 (&x)[4], const Guard& g) {
  const f8::Rows<__nv_bfloat16> m(base, rows, ld, cols, g);
  f8::store_chunk<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16*>(base) + row * ld + col, &x[0].x, n, m);
}

// ACT: the activation (one kernel for each: the branch around eight values' work cost as much as the work).  VEC: chunks of 8
// columns can be read and written at once (but for one that a row ends in).
template <int ACT, bool GATED, bool CODES, bool VEC, bool SUMS>
__global__ void __launch_bounds__(kThreads, VEC ? 3 : 2) linear_grad_kernel(const __grid_constant__ LinearGradParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lanes = p.strip / 8, at = (int)threadIdx.x % lanes, step = kThreads / lanes;  // (8 or 32 threads to a row)
  const int col = (int)blockIdx.x * p.strip + 8 * at;
  const int n = max(0, min(8, p.cols - col));
  const int64_t r0 = p.rows * blockIdx.y / p.row_blocks + threadIdx.x / lanes, r1 = p.rows * (blockIdx.y + 1) / p.row_blocks;
  const LinearKeptIn y{p.dy, nullptr, p.lddy, 0, 0};
  constexpr bool kAct = ACT != SGEMM_ACT_NONE || GATED;  // A is read
  float2 sum[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
  // the work on 8 values of row r
  const auto work = [&](auto vec, int64_t row, const float2 (&g)[4], const float2 (&x)[4], const float2 (&u)[4]) {
    constexpr bool kVec = decltype(vec)::value;
    float2 d[4];
    if constexpr (GATED) {
      float2 du[4], h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 f, df;
        act_grad<ACT>(x[e], f, df);
        d[e] = mul(mul(g[e], u[e]), df);
        du[e] = mul(g[e], f);
        h[e] = mul(f, u[e]);
      }
      if (p.da) {
        put8<kVec>(p.da, p.ldd, p.rows, p.cols, row, col, n, d, p.guard);
        put8<kVec>(p.db, p.ldd, p.rows, p.cols, row, col, n, du, p.guard);
      }
      if (p.h) put8<kVec>(p.h, p.ldh, p.rows, p.cols, row, col, n, h, p.guard);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 f, df;
        if (kAct) act_grad<ACT>(x[e], f, df);
        d[e] = kAct ? mul(g[e], df) : g[e];
        if (SUMS) sum[e] = add(sum[e], d[e]);
      }
      if (p.da) put8<kVec>(p.da, p.ldd, p.rows, p.cols, row, col, n, d, p.guard);
    }
  };
  if constexpr (VEC) {
    struct None {};
    __shared__ KeptRing<false> ring_y;
    __shared__ typename std::conditional<kAct, KeptRing<CODES>, None>::type ring_a;
    __shared__ typename std::conditional<GATED, KeptRing<CODES>, None>::type ring_b;
    if (n == 8) {
      const auto copy = [&](int s, int64_t row) {
        if (row < r1) {
          ring_y.copy(s, y, p.rows, p.cols, row, col, p.guard);
          if constexpr (kAct) ring_a.copy(s, p.a, p.rows, p.cols, row, col, p.guard);
          if constexpr (GATED) ring_b.copy(s, p.b, p.rows, p.cols, row, col, p.guard);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int s = 0; s < kStages; ++s) copy(s, r0 + s * step);
      int s = 0;
      for (int64_t row = r0; row < r1; row += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        float2 g[4], x[4], u[4];
        ring_y.get(s, g);
        if constexpr (kAct) ring_a.get(s, x);
        if constexpr (GATED) ring_b.get(s, u);
        work(std::true_type{}, row, g, x, u);
        copy(s, row + kStages * step);
        s = s + 1 == kStages ? 0 : s + 1;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  }
  if (VEC ? n > 0 && n < 8 : n > 0) {
    for (int64_t r = r0; r < r1; r += kBatch * step) {
      KeptLoad<false> dy[kBatch];
      KeptLoad<CODES> a[kBatch], b[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool there = r + k * step < r1;
        const int64_t row = there ? r + k * step : r;
        const int here = there ? n : 0;
        dy[k].load(y, p.rows, p.cols, row, col, here, p.guard);
        if (kAct) a[k].load(p.a, p.rows, p.cols, row, col, here, p.guard);
        if (GATED) b[k].load(p.b, p.rows, p.cols, row, col, here, p.guard);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (r + k * step >= r1) break;
        float2 g[4], x[4], u[4];
        dy[k].get(g);
        if (kAct) a[k].get(x);
        if (GATED) b[k].get(u);
        work(std::false_type{}, r + k * step, g, x, u);
      }
    }
  }
  if constexpr (SUMS) {
    __shared__ __align__(16) float warps[kThreads / 32][kWide];
    __shared__ float strip[kWide];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (lanes == 8)  // over the warp's four rows
#pragma unroll
        for (int m = 8; m < 32; m *= 2)
          sum[e] = add(sum[e], make_float2(__shfl_xor_sync(0xffffffffu, sum[e].x, m), __shfl_xor_sync(0xffffffffu, sum[e].y, m)));
      if ((int)threadIdx.x % 32 < lanes) *reinterpret_cast<float2*>(&warps[threadIdx.x / 32][8 * at + 2 * e]) = sum[e];
    }
    __syncthreads();
    const int c = (int)blockIdx.x * p.strip + (int)threadIdx.x;
    const bool mine = (int)threadIdx.x < p.strip && c < p.cols;
    float s = 0.0f;
    if (mine) {
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) s += warps[w][threadIdx.x];
      strip[threadIdx.x] = s;
      if (p.partial) put_at(p.guard, f8::kSitePart, p.partial, (int64_t)blockIdx.y * p.cols + c, (int64_t)p.row_blocks * p.cols, s);
    }
    if (p.partial) return;
    tc::cluster_sync();
    if (blockIdx.y == 0 && mine) {
      for (int k = 1; k < p.row_blocks; ++k) {  // (the row blocks are the cluster)
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::map_to_rank(smem_addr(&strip[threadIdx.x]), (uint32_t)k)) : "memory");
        s += v;
      }
      put_at(p.guard, f8::kSiteOut, p.dbias, c, p.cols, s);
    }
    tc::cluster_sync();  // no CTA leaves while its sums may be read
  }
}

// dbias from the row blocks' sums: a column per lane, the warps share the blocks.
__global__ void __launch_bounds__(kThreads) linear_bias_kernel(const __grid_constant__ LinearGradParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kWarps = kThreads / 32;
  __shared__ float part[kWarps][32];
  const int warp = (int)threadIdx.x / 32, lane = (int)threadIdx.x % 32, c = (int)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < p.cols)
#pragma unroll 4
    for (int b = warp; b < p.row_blocks; b += kWarps)
      s += get_at(p.guard, f8::kSitePart, p.partial, (int64_t)b * p.cols + c, (int64_t)p.row_blocks * p.cols);
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.cols) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][lane];
    put_at(p.guard, f8::kSiteOut, p.dbias, c, p.cols, s);
  }
}

// Up to three matrices one behind the other, in chunks of 8 columns (codes are read one by one, at any alignment: 8192 x 4096 of them
// take 30 us, 3.4 TB/s).
__global__ void __launch_bounds__(kThreads) linear_expand_kernel(const __grid_constant__ LinearExpandParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int which = 0;
  int64_t block = blockIdx.x;
  while (block >= p.part[which].blocks) block -= p.part[which++].blocks;
  const LinearExpand& m = p.part[which];
  const int chunks = (m.cols + 7) / 8;
  const int64_t total = m.rows * chunks;
  const auto run = [&](auto codes) {
    constexpr int kChunks = kExpandChunks;
    KeptLoad<decltype(codes)::value> v[kChunks];
    int64_t row[kChunks];
    int col[kChunks], n[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int64_t i = (block * kChunks + k) * kThreads + threadIdx.x, j = i < total ? i : 0;
      row[k] = total <= 0x7fffffff ? (uint32_t)j / (uint32_t)chunks : j / chunks;
      col[k] = (int)(j - row[k] * chunks) * 8;
      n[k] = i < total ? min(8, m.cols - col[k]) : 0;
      v[k].load(m.m, m.rows, m.cols, row[k], col[k], n[k], p.guard);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      float2 x[4];
      v[k].get(x);
      // (whole chunks: rows of the copy have room for them, and nothing reads behind their ends)
      if (n[k] > 0 && in_range(p.guard.fault, p.guard.word, f8::kSitePart, row[k] * m.ldd + col[k], 8, m.rows * m.ldd)) {
        Chunk<__nv_bfloat16> c;
        c.put(&x[0].x);
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(m.dst) + row[k] * m.ldd + col[k]) = c.raw;
      }
    }
  };
  if (m.m.scale) run(std::true_type{});
  else           run(std::false_type{});
}

template <typename P>
cudaError_t launch(void (*kernel)(P), dim3 grid, int cluster_y, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = (unsigned)cluster_y;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster_y > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool GATED, bool CODES, bool VEC, bool SUMS>
cudaError_t launch_act(const LinearGradParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.cols + p.strip - 1) / p.strip), (unsigned)p.row_blocks);
  cudaError_t e = cudaErrorInvalidValue;
  with_act(p.act, [&](auto act) { e = launch(linear_grad_kernel<decltype(act)::value, GATED, CODES, VEC, SUMS>, grid, SUMS && !p.partial ? p.row_blocks : 1, p, stream); });
  if (SUMS && p.partial && e == cudaSuccess) e = launch(linear_bias_kernel, dim3((unsigned)((p.cols + 31) / 32)), 1, p, stream);
  return e;
}
template <bool VEC>
cudaError_t launch_form(const LinearGradParams& p, cudaStream_t stream) {
  const bool codes = p.a.scale != nullptr;
  if (p.b.data) return codes ? launch_act<true, true, VEC, false>(p, stream) : launch_act<true, false, VEC, false>(p, stream);
  if (p.dbias) return codes ? launch_act<false, true, VEC, true>(p, stream) : launch_act<false, false, VEC, true>(p, stream);
  return codes ? launch_act<false, true, VEC, false>(p, stream) : launch_act<false, false, VEC, false>(p, stream);
}

}  // namespace
}  // namespace lin

void shape_linear_grad(LinearGradParams* p, bool clusters, int sm_count) {
  // strips of 512 bytes of a row (64 of 128 bytes read and wrote at half the memory's rate in the gated form), or of 128 bytes
  // where there would be too few of them
  const int64_t wide = (p->cols + lin::kWide - 1) / lin::kWide, most = (p->rows + 31) / 32;
  p->strip = wide * std::min<int64_t>(8, most) >= sm_count ? lin::kWide : lin::kNarrow;
  const int64_t strips = (p->cols + p->strip - 1) / p->strip;
  const bool narrow = p->strip == lin::kNarrow;
  int n = clusters ? 8 : 1;  // a cluster's CTAs
  while (n > 1 && n > most) n /= 2;
  // Clusters that leave room on the SMs cost more than a second kernel from some rows on: 1 us or so on the GPU, and 4 us of the
  // host, which a call of fewer rows would wait for.  Joined and by a second kernel, us of the pass alone: GELU 16384 rows 64 columns 20.9
  // and 6.7, 1216 columns 49 and 26, 2048 columns 52 and 33, 4096 columns 8192 rows 44 and 34; without an activation 65536 rows 64 columns
  // 33 and 6.9, 512 columns 40 and 15.  (600 rows of 256 columns, whole calls of 256 inputs: 28 joined and 31.)
  const bool act = p->act != SGEMM_ACT_NONE;
  const bool few = strips * n < (act ? 4 : 2) * sm_count && p->rows > (act ? 8192 : 32768);
  p->joined = p->dbias && narrow && !few;
  if (p->joined) {
    p->row_blocks = n;
  } else {
    // CTAs of no fewer than 32 rows, eight per SM; where a second kernel adds the sums of narrow strips, which has little to read
    // per row block but a wait for each few of them, two, or with an activation's work at least an eighth as many row blocks as SMs
    int64_t want = ((p->dbias && narrow ? 2 : 8) * (int64_t)sm_count + strips - 1) / strips;
    if (p->dbias && narrow && act) want = std::max<int64_t>(want, sm_count / 8);
    p->row_blocks = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(want, most), 65535));
  }
}

cudaError_t launch_linear_grad(const LinearGradParams& p, cudaStream_t stream) {
  return p.vec ? lin::launch_form<true>(p, stream) : lin::launch_form<false>(p, stream);
}

cudaError_t launch_linear_expand(LinearExpandParams& p, cudaStream_t stream) {
  int64_t blocks = 0;
  for (LinearExpand& m : p.part) {
    m.blocks = (m.rows * ((m.cols + 7) / 8) + lin::kExpandChunks * lin::kThreads - 1) / (lin::kExpandChunks * lin::kThreads);
    blocks += m.blocks;
  }
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return lin::launch(lin::linear_expand_kernel, dim3((unsigned)blocks), 1, p, stream);
}

}  // namespace sgemm_impl
