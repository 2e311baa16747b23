// kernel_linear_grad.cu -- the elementwise part of the backward passes of a layer and of a gated block, for sm_103a, and the
// aligned BF16 copies of operands that the tensor cores' loads cannot read as they are.
//
//     layer:  dA = dY * act'(A),  dbias = sum over the rows of dA
//     gated:  dA = dH * B * act'(A),  dB = dH * act(A),  H = act(A) * B
//
// A and B as the forward pass kept them: BF16, or 8-bit codes times the scale of their group of 128.  One pass over the data,
// bound by the memory and nearly as much by the instructions of an activation's derivative (two values at a time in packed
// arithmetic).  A thread takes 8 columns of a row (16 bytes of BF16, 8 of codes), eight threads a line of 128 bytes, and has all
// its loads of two rows on their way before either is used.  Column sums are held per thread in FP32, joined within the CTA and
// then by a cluster of up to 8 CTAs that share the rows of a strip of 64 columns, both in a fixed order: no second kernel.
#include "linear_common.cuh"

namespace sgemm_impl {
namespace lin {
namespace {

constexpr int kThreads = 256, kStrip = 64, kLanes = kStrip / 8, kRowLanes = kThreads / kLanes;
constexpr int kBatch = 2;         // rows whose loads are on their way together
constexpr int kExpandChunks = 4;  // the same of the copies, in chunks of 8 columns

// 8 consecutive values, n of them there, sent for and then waited for.  VEC: n is 8 or 0, and they can be read at once.
template <bool CODES, bool VEC>
struct KeptLoad;
template <bool VEC>
struct KeptLoad<false, VEC> {
  f8::Loading<__nv_bfloat16, VEC> v;
  __device__ __forceinline__ void load(const LinearKeptIn& k, int64_t rows, int cols, int64_t row, int col, int n, const Guard& g) {
    const f8::Rows<__nv_bfloat16> m(k.data, rows, k.ld, cols, g);
    v.load(m.base + row * k.ld + col, n, m);
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const { v.get().get(&x[0].x); }
};
template <bool VEC>
struct KeptLoad<true, VEC> {
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
    if (VEC) {
      c = *reinterpret_cast<const uint2*>(base + at);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) (e < 4 ? c.x : c.y) |= (uint32_t)base[at + e] << (8 * (e % 4));
    }
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((e < 2 ? c.x : c.y) >> (16 * (e % 2))), __NV_E4M3);
      x[e] = mul(__half22float2(__half2(h)), both(s));
    }
  }
};

// 8 values as BF16, n of them there, to a row of an aligned (VEC) or any other matrix.
template <bool VEC>
__device__ __forceinline__ void put8(void* base, int64_t ld, int64_t rows, int cols, int64_t row, int col, int n, const float2 (&x)[4], const Guard& g) {
  const f8::Rows<__nv_bfloat16> m(base, rows, ld, cols, g);
  f8::store_chunk<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16*>(base) + row * ld + col, &x[0].x, n, m);
}

// ACT: the activation (one kernel for each: the branch around eight values' work cost as much as the work).
template <int ACT, bool GATED, bool CODES, bool VEC, bool SUMS>
__global__ void __launch_bounds__(kThreads) linear_grad_kernel(const __grid_constant__ LinearGradParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int col = (int)blockIdx.x * kStrip + 8 * (int)(threadIdx.x % kLanes);
  const int n = max(0, min(8, p.cols - col));
  const int64_t r0 = p.rows * blockIdx.y / p.row_blocks, r1 = p.rows * (blockIdx.y + 1) / p.row_blocks;
  const LinearKeptIn y{p.dy, nullptr, p.lddy, 0, 0};
  constexpr bool kAct = ACT != SGEMM_ACT_NONE || GATED;  // A is read
  float2 sum[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
  if (n > 0) {
    for (int64_t r = r0 + threadIdx.x / kLanes; r < r1; r += kBatch * kRowLanes) {
      KeptLoad<false, VEC> dy[kBatch];
      KeptLoad<CODES, VEC> a[kBatch], b[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool there = r + k * kRowLanes < r1;
        const int64_t row = there ? r + k * kRowLanes : r;
        const int here = there ? n : 0;
        dy[k].load(y, p.rows, p.cols, row, col, here, p.guard);
        if (kAct) a[k].load(p.a, p.rows, p.cols, row, col, here, p.guard);
        if (GATED) b[k].load(p.b, p.rows, p.cols, row, col, here, p.guard);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t row = r + k * kRowLanes;
        if (row >= r1) break;
        float2 g[4], x[4], d[4];
        dy[k].get(g);
        if (kAct) a[k].get(x);
        if (GATED) {
          float2 u[4], du[4], h[4];
          b[k].get(u);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 f, df;
            act_grad<ACT>(x[e], f, df);
            d[e] = mul(mul(g[e], u[e]), df);
            du[e] = mul(g[e], f);
            h[e] = mul(f, u[e]);
          }
          if (p.da) {
            put8<VEC>(p.da, p.ldd, p.rows, p.cols, row, col, n, d, p.guard);
            put8<VEC>(p.db, p.ldd, p.rows, p.cols, row, col, n, du, p.guard);
          }
          if (p.h) put8<VEC>(p.h, p.ldh, p.rows, p.cols, row, col, n, h, p.guard);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 f, df;
            if (kAct) act_grad<ACT>(x[e], f, df);
            d[e] = kAct ? mul(g[e], df) : g[e];
            if (SUMS) sum[e] = add(sum[e], d[e]);
          }
          if (p.da) put8<VEC>(p.da, p.ldd, p.rows, p.cols, row, col, n, d, p.guard);
        }
      }
    }
  }
  if constexpr (SUMS) {
    __shared__ float warps[kThreads / 32][kStrip], strip[kStrip];
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // over the warp's four rows
#pragma unroll
      for (int m = kLanes; m < 32; m *= 2)
        sum[e] = add(sum[e], make_float2(__shfl_xor_sync(0xffffffffu, sum[e].x, m), __shfl_xor_sync(0xffffffffu, sum[e].y, m)));
      if (threadIdx.x % 32 < kLanes) *reinterpret_cast<float2*>(&warps[threadIdx.x / 32][8 * (threadIdx.x % kLanes) + 2 * e]) = sum[e];
    }
    __syncthreads();
    float s = 0.0f;
    if (threadIdx.x < kStrip) {
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) s += warps[w][threadIdx.x];
      strip[threadIdx.x] = s;
    }
    const int c = (int)blockIdx.x * kStrip + (int)threadIdx.x;
    tc::cluster_sync();
    if (blockIdx.y == 0 && threadIdx.x < kStrip && c < p.cols) {
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

// Up to three matrices one behind the other, in chunks of 8 columns.
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
    KeptLoad<decltype(codes)::value, false> v[kChunks];
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
  const dim3 grid((unsigned)((p.cols + kStrip - 1) / kStrip), (unsigned)p.row_blocks);
  cudaError_t e = cudaErrorInvalidValue;
  with_act(p.act, [&](auto act) { e = launch(linear_grad_kernel<decltype(act)::value, GATED, CODES, VEC, SUMS>, grid, SUMS ? p.row_blocks : 1, p, stream); });
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

int linear_grad_row_blocks(int64_t rows, int cols, bool sums, bool clusters, int sm_count) {
  if (sums && !clusters) return 1;
  const int64_t strips = (cols + lin::kStrip - 1) / lin::kStrip;
  // eight CTAs per SM, of no fewer rows than two batches
  const int64_t want = (8 * (int64_t)sm_count + strips - 1) / strips, most = (rows + 2 * lin::kBatch * lin::kRowLanes - 1) / (2 * lin::kBatch * lin::kRowLanes);
  int64_t blocks = want < most ? want : most;
  if (!sums) return (int)(blocks < 1 ? 1 : blocks > 65535 ? 65535 : blocks);
  int n = 8;  // a cluster
  while (n > 1 && n > most) n /= 2;
  return n;
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
