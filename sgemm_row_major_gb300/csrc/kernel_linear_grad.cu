// kernel_linear_grad.cu -- the elementwise part of the backward passes of a layer and of a gated block, for sm_103a, and the
// aligned BF16 copies of operands that the tensor cores' loads cannot read as they are.
//
//     layer:  dA = dY * act'(A),  dbias = sum over the rows of dA
//     gated:  dA = dH * B * act'(A),  dB = dH * act(A),  H = act(A) * B
//
// A and B as the forward pass kept them: BF16, or 8-bit codes times the scale of their group of 128.  One pass over the data,
// bound by the memory; a thread takes 8 columns of a row (16 bytes of BF16, 8 of codes), and rows 8 apart with all its loads
// of two rows on their way before either is used.  Column sums are held per thread in FP32 over the rows of a block, joined in
// shared memory in a fixed order, and the blocks' sums are added by a second kernel in a fixed order.
#include "linear_common.cuh"

namespace sgemm_impl {
namespace lin {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kStrip = 256;  // columns of a CTA: 8 per lane

// 8 consecutive values of a kept matrix, sent for and then waited for.
template <bool CODES>
struct KeptLoad;
template <>
struct KeptLoad<false> {
  f8::Loading<__nv_bfloat16, true> v;
  f8::Loading<__nv_bfloat16, false> u;
  bool vec;
  __device__ __forceinline__ void load(const LinearKeptIn& k, int64_t rows, int cols, int64_t row, int col, int n, const Guard& g) {
    const f8::Rows<__nv_bfloat16> m(k.data, rows, k.ld, cols, g);
    const __nv_bfloat16* p = m.base + row * k.ld + col;
    vec = k.vec && n == 8;
    if (vec) v.load(p, 8, m);
    else     u.load(p, n, m);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if (vec) v.get().get(x);
    else     u.get().get(x);
  }
};
template <>
struct KeptLoad<true> {
  uint32_t c[2];
  float s;
  __device__ __forceinline__ void load(const LinearKeptIn& k, int64_t rows, int cols, int64_t row, int col, int n, const Guard& g) {
    c[0] = c[1] = 0u;
    s = 0.0f;
    if (n <= 0) return;
    const uint8_t* base = static_cast<const uint8_t*>(k.data);
    const int64_t at = row * k.ld + col;
    if (!in_range(g.fault, g.word, f8::kSiteCodes, at, n, extent(rows, k.ld, cols))) return;
    s = get_at(g, f8::kSiteScale, k.scale, row * k.lds + (col >> 7), extent(rows, k.lds, (cols + 127) / 128));
    if (k.vec && n == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(base + at);
      c[0] = u.x;
      c[1] = u.y;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) c[e / 4] |= (uint32_t)base[at + e] << (8 * (e % 4));
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c[e / 2] >> (16 * (e % 2))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      x[2 * e] = f.x * s;
      x[2 * e + 1] = f.y * s;
    }
  }
};

// 8 values of BF16, n of them there, to a row of an aligned (VEC) or any other matrix.
__device__ __forceinline__ void put8(void* base, int64_t ld, int64_t rows, int cols, int64_t row, int col, int n, bool vec, const float (&x)[8],
                                     const Guard& g) {
  const f8::Rows<__nv_bfloat16> m(base, rows, ld, cols, g);
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + row * ld + col;
  if (vec && n == 8) f8::store_chunk<__nv_bfloat16, true>(p, x, 8, m);
  else               f8::store_chunk<__nv_bfloat16, false>(p, x, n, m);
}

template <bool GATED, bool CODES, bool SUMS>
__global__ void __launch_bounds__(kThreads) linear_grad_kernel(const LinearGradParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kRows = 2;  // whose loads are on their way together
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = (int)blockIdx.x * kStrip + 8 * lane;
  const int n = max(0, min(8, p.cols - col));
  const int64_t r0 = p.rows * blockIdx.y / p.row_blocks, r1 = p.rows * (blockIdx.y + 1) / p.row_blocks;
  float sum[SUMS ? 8 : 1];
#pragma unroll
  for (int e = 0; e < (SUMS ? 8 : 1); ++e) sum[e] = 0.0f;
  if (n > 0) {
    for (int64_t r = r0 + warp; r < r1; r += kRows * kWarps) {
      KeptLoad<false> dy[kRows];
      KeptLoad<CODES> a[kRows], b[GATED ? kRows : 1];
      const LinearKeptIn y{p.dy, nullptr, p.lddy, 0, p.dy_vec};
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t row = r + k * kWarps;
        const int here = row < r1 ? n : 0;
        const int64_t at = row < r1 ? row : r;
        dy[k].load(y, p.rows, p.cols, at, col, here, p.guard);
        if (GATED || p.a.data) a[k].load(p.a, p.rows, p.cols, at, col, here, p.guard);
        if (GATED) b[GATED ? k : 0].load(p.b, p.rows, p.cols, at, col, here, p.guard);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t row = r + k * kWarps;
        if (row >= r1) break;
        float g[8], x[8], d[8];
        dy[k].get(g);
        if (GATED) {
          float u[8], du[8], h[8];
          a[k].get(x);
          b[GATED ? k : 0].get(u);
          with_act(p.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 ge = make_float2(g[e], g[e + 1]), ue = make_float2(u[e], u[e + 1]);
              float2 f, df;
              act_grad<decltype(act)::value>(make_float2(x[e], x[e + 1]), f, df);
              *reinterpret_cast<float2*>(&d[e]) = mul(mul(ge, ue), df);
              *reinterpret_cast<float2*>(&du[e]) = mul(ge, f);
              *reinterpret_cast<float2*>(&h[e]) = mul(f, ue);
            }
          });
          if (p.da) {
            put8(p.da, p.ldd, p.rows, p.cols, row, col, n, true, d, p.guard);
            put8(p.db, p.ldd, p.rows, p.cols, row, col, n, true, du, p.guard);
          }
          if (p.h) put8(p.h, p.ldh, p.rows, p.cols, row, col, n, p.h_vec, h, p.guard);
        } else {
          if (p.a.data) {
            a[k].get(x);
            with_act(p.act, [&](auto act) {
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                float2 f, df;
                act_grad<decltype(act)::value>(make_float2(x[e], x[e + 1]), f, df);
                *reinterpret_cast<float2*>(&d[e]) = mul(make_float2(g[e], g[e + 1]), df);
              }
            });
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = g[e];
          }
          if (p.da) put8(p.da, p.ldd, p.rows, p.cols, row, col, n, true, d, p.guard);
          if (SUMS) {
#pragma unroll
            for (int e = 0; e < (SUMS ? 8 : 1); ++e) sum[e] += d[e];
          }
        }
      }
    }
  }
  if constexpr (SUMS) {
    __shared__ float part[kWarps][kStrip];
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][8 * lane + e] = sum[e];
    __syncthreads();
    const int c = (int)blockIdx.x * kStrip + (int)threadIdx.x;
    if (c < p.cols) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
      if (p.row_blocks == 1) put_at(p.guard, f8::kSiteOut, p.dbias, c, p.cols, s);
      else put_at(p.guard, f8::kSitePart, p.partial, (int64_t)blockIdx.y * p.cols + c, (int64_t)p.row_blocks * p.cols, s);
    }
  }
}

// dbias from the row blocks' sums, a column per lane, 8 warps over the blocks.
__global__ void __launch_bounds__(kThreads) linear_bias_kernel(const LinearGradParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float part[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = (int)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < p.cols)
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

template <bool CODES>
__global__ void __launch_bounds__(kThreads) linear_expand_kernel(const LinearKeptIn m, int64_t rows, int cols, void* dst, int64_t ldd,
                                                                 const Guard guard) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int chunks = (cols + 7) / 8;
  const int64_t total = rows * chunks, step = (int64_t)gridDim.x * kThreads;
  constexpr int kBatch = 4;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += kBatch * step) {
    KeptLoad<CODES> v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t j = i + k * step, row = j < total ? j / chunks : 0;
      const int col = (int)(j - row * chunks) * 8;
      v[k].load(m, rows, cols, row, j < total ? col : 0, j < total ? min(8, cols - col) : 0, guard);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t j = i + k * step;
      if (j >= total) break;
      const int64_t row = j / chunks;
      const int col = (int)(j - row * chunks) * 8;
      float x[8];
      v[k].get(x);
      put8(dst, ldd, rows, cols, row, col, min(8, cols - col), true, x, guard);
    }
  }
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace lin

int linear_grad_row_blocks(int64_t rows, int cols, int sm_count) {
  // four CTAs per SM, no fewer than 32 rows each
  const int64_t strips = (cols + lin::kStrip - 1) / lin::kStrip;
  int64_t blocks = (8 * (int64_t)sm_count + strips - 1) / strips;
  if (blocks > (rows + 31) / 32) blocks = (rows + 31) / 32;
  return (int)(blocks < 1 ? 1 : blocks > 65535 ? 65535 : blocks);
}

cudaError_t launch_linear_grad(const LinearGradParams& p, cudaStream_t stream) {
  using namespace lin;
  const dim3 grid((unsigned)((p.cols + kStrip - 1) / kStrip), (unsigned)p.row_blocks);
  const bool codes = p.a.scale != nullptr, sums = p.dbias != nullptr;
  cudaError_t e;
  if (p.b.data) e = launch(codes ? linear_grad_kernel<true, true, false> : linear_grad_kernel<true, false, false>, grid, stream, p);
  else if (sums) e = launch(codes ? linear_grad_kernel<false, true, true> : linear_grad_kernel<false, false, true>, grid, stream, p);
  else e = launch(codes ? linear_grad_kernel<false, true, false> : linear_grad_kernel<false, false, false>, grid, stream, p);
  if (e == cudaSuccess && sums && p.row_blocks > 1) e = launch(linear_bias_kernel, dim3((unsigned)((p.cols + 31) / 32)), stream, p);
  return e;
}

cudaError_t launch_linear_expand(const LinearKeptIn& m, int64_t rows, int64_t cols, void* dst, int64_t ldd, const Guard& guard,
                                 cudaStream_t stream) {
  const int64_t blocks = (rows * ((cols + 7) / 8) + 4 * lin::kThreads - 1) / (4 * lin::kThreads);
  const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
  return lin::launch(m.scale ? lin::linear_expand_kernel<true> : lin::linear_expand_kernel<false>, grid, stream, m, rows, (int)cols, dst, ldd,
                     guard);
}

}  // namespace sgemm_impl
