// kernel_fp8_norm.cu -- RMS norm with residual addition and 8-bit output, and its gradients.
//
// Forward, for a row of n columns:   h = x + r,  rstd = (sum h^2 / n + eps)^(-1/2),  y = h rstd w,
// and y in E4M3 codes with a scale per 128 columns.  One CTA per row: a thread keeps its 8-column
// chunks of h in registers between the sum and the output, so x and r are read once and h and the
// codes written once (an HBM stream: 7 bytes per element of a BF16 row with a residual).  16
// neighbouring threads hold one group of 128 columns, so a group's largest value is a shuffle away.
//
// Backward:   dx = rstd (dy w - h rstd^2 mean(dy w h)) + dh,   dw = sum_rows dy h rstd.
// A persistent grid: a CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ..., its threads own
// fixed columns and keep their part of dw in registers (the wide form: in shared memory), so dw
// costs no traffic per row; the CTAs' sums go to `partial` and a second kernel adds them in CTA
// order.  The next row's chunks are loaded before the current row's sum is waited for.
#include <algorithm>

#include "fp8_common.cuh"
#include "fp8_internal.h"

namespace sgemm_impl {
namespace f8 {
namespace {

constexpr int kChunk = 8;         // columns a thread takes at a time
constexpr int kMaxWarps = 32;

// 8 columns as stored: one 16-byte vector of BF16, two of FP32.
template <typename T>
struct Chunk8 {
  static constexpr int kVecs = kChunk / Chunk<T>::V;
  Chunk<T> c[kVecs];
  __device__ __forceinline__ void load(const T* p, int n, bool vec) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) c[i] = load_chunk(p + i * Chunk<T>::V, (int64_t)(n - i * Chunk<T>::V), vec);
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) c[i].get(v + i * Chunk<T>::V);
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v, int n, bool vec) {
#pragma unroll
  for (int i = 0; i < kChunk / Chunk<T>::V; ++i)
    store_chunk(p + i * Chunk<T>::V, v + i * Chunk<T>::V, (int64_t)(n - i * Chunk<T>::V), vec);
}

// Sum over the CTA of one float per thread; `slot` is used by one call at a time.
__device__ __forceinline__ float cta_sum(float v, float* slot) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < (int)(blockDim.x >> 5) ? slot[lane] : 0.0f);
}

// y of one chunk (columns col .. col + 7 of row `row`) to the outputs that are wanted.
template <typename T>
__device__ __forceinline__ void emit(const NormParams& p, int64_t row, int col, const float* h, float rstd) {
  const int left = p.cols - col;
  const bool vec = p.vec != 0;
  float y[kChunk];
  {
    Chunk8<T> w;
    w.load(static_cast<const T*>(p.w) + col, left, vec);
    w.get(y);
  }
#pragma unroll
  for (int e = 0; e < kChunk; ++e) y[e] = h[e] * rstd * y[e];  // columns past the end: h = 0
  if (p.y && left > 0) store8(static_cast<T*>(p.y) + row * p.ldy + col, y, left, vec);
  if (p.q) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) m = fmaxf(m, finite_abs(y[e]));
    const float s = group_scale(lanes_max<16>(m), kMaxE4M3);
    if (left > 0) {
      if (col % 128 == 0) p.s[row * p.lds + col / 128] = s;
      float inv[kChunk];
#pragma unroll
      for (int e = 0; e < kChunk; ++e) inv[e] = __frcp_rn(s);
      store_codes<kChunk, true>(p.q + row * p.ldq + col, y, inv, left, vec, false);
    }
  }
}

template <typename T>
__device__ __forceinline__ void load_h(const NormParams& p, int64_t row, int col, float* h) {
  const int left = p.cols - col;
  const bool vec = p.vec != 0;
  Chunk8<T> x;
  x.load(static_cast<const T*>(p.x) + row * p.ldx + col, left, vec);
  if (p.r) {
    Chunk8<T> r;
    r.load(static_cast<const T*>(p.r) + row * p.ldr + col, left, vec);
    float b[kChunk];
    x.get(h);
    r.get(b);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) h[e] += b[e];
  } else {
    x.get(h);
  }
}

// NV chunks per thread; chunk j of thread t is columns 8 (j blockDim.x + t) .. + 7.
template <typename T, int NV>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormParams p) {
  __shared__ float slot[kMaxWarps];
  const int64_t row = blockIdx.x;
  float h[NV][kChunk];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) load_h<T>(p, row, kChunk * (j * (int)blockDim.x + (int)threadIdx.x), h[j]);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) a = fmaf(h[j][e], h[j][e], a);
    ss += a;
  }
  const float rstd = __frsqrt_rn(cta_sum(ss, slot) / (float)p.cols + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x);
    if (p.h && col < p.cols) store8(static_cast<T*>(p.h) + row * p.ldh + col, h[j], p.cols - col, p.vec != 0);
    emit<T>(p, row, col, h[j], rstd);
  }
}

// Rows too long for registers: a second pass reads x and r again (from L2) for the output.
template <typename T>
__global__ void __launch_bounds__(1024) rmsnorm_wide_kernel(const NormParams p) {
  __shared__ float slot[kMaxWarps];
  const int64_t row = blockIdx.x;
  const int step = kChunk * (int)blockDim.x;
  float ss = 0.0f;
  for (int64_t c0 = 0; c0 < p.cols; c0 += step) {  // 64-bit: c0 + step may pass 2^31
    float h[kChunk];
    const int64_t col = c0 + kChunk * (int)threadIdx.x;
    if (col >= p.cols) continue;
    load_h<T>(p, row, (int)col, h);
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) a = fmaf(h[e], h[e], a);
    ss += a;
  }
  const float rstd = __frsqrt_rn(cta_sum(ss, slot) / (float)p.cols + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  for (int64_t c0 = 0; c0 < p.cols; c0 += step) {
    float h[kChunk];
    // every lane stays in the loop (the groups' shuffles); past the end it works on no columns
    const int col = (int)min(c0 + kChunk * (int)threadIdx.x, ((int64_t)p.cols + 7) / 8 * 8);
    load_h<T>(p, row, col, h);
    // h may overwrite x or r: only this thread reads these columns, and it has
    if (p.h && col < p.cols) store8(static_cast<T*>(p.h) + row * p.ldh + col, h, p.cols - col, p.vec != 0);
    emit<T>(p, row, col, h, rstd);
  }
}

constexpr int kRegCols = 32768;  // 1024 threads x 4 chunks

template <typename T>
cudaError_t launch_forward(const NormParams& p, cudaStream_t stream) {
  const int chunks = (int)(((int64_t)p.cols + kChunk - 1) / kChunk);
  const dim3 grid((unsigned)p.rows);
  // two chunks per thread (four beyond 8192 columns, where 1024 threads would need them anyway)
  const auto threads = [&](int nv) { return std::min(1024, (chunks + 32 * nv - 1) / (32 * nv) * 32); };
  if (p.cols > kRegCols) rmsnorm_wide_kernel<T><<<grid, 1024, 0, stream>>>(p);
  else if (chunks <= 128) rmsnorm_kernel<T, 1><<<grid, threads(1), 0, stream>>>(p);
  else if (chunks <= 1024) rmsnorm_kernel<T, 2><<<grid, threads(2), 0, stream>>>(p);
  else rmsnorm_kernel<T, 4><<<grid, threads(4), 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ backward

template <typename T, int NV>
struct GradRow {  // a thread's chunks of dy, h and dh of one row
  Chunk8<T> dy[NV], h[NV], dh[NV];
  float rstd;
  __device__ __forceinline__ void load(const NormGradParams& p, int64_t row) {
    rstd = p.rstd[row];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x), left = p.cols - col;
      dy[j].load(static_cast<const T*>(p.dy) + row * p.lddy + col, left, p.vec != 0);
      h[j].load(static_cast<const T*>(p.h) + row * p.ldh + col, left, p.vec != 0);
      if (p.dh) dh[j].load(static_cast<const T*>(p.dh) + row * p.lddh + col, left, p.vec != 0);
    }
  }
};

// One chunk of dx, and its part of dw added to acc.
template <typename T>
__device__ __forceinline__ void grad_chunk(const NormGradParams& p, int64_t row, int col, const Chunk8<T>& cdy,
                                           const Chunk8<T>& ch, const Chunk8<T>& cdh, const float* w, float rstd,
                                           float c, float* acc) {
  float dy[kChunk], h[kChunk], dx[kChunk];
  cdy.get(dy);
  ch.get(h);
#pragma unroll
  for (int e = 0; e < kChunk; ++e) {
    acc[e] = fmaf(dy[e] * h[e], rstd, acc[e]);
    dx[e] = rstd * (dy[e] * w[e] - h[e] * c);
  }
  if (p.dh) {
    float dh[kChunk];
    cdh.get(dh);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) dx[e] += dh[e];
  }
  if (col < p.cols) store8(static_cast<T*>(p.dx) + row * p.lddx + col, dx, p.cols - col, p.vec != 0);
}

template <typename T>
__device__ __forceinline__ float grad_dot(const Chunk8<T>& cdy, const Chunk8<T>& ch, const float* w) {
  float dy[kChunk], h[kChunk], a = 0.0f;
  cdy.get(dy);
  ch.get(h);
#pragma unroll
  for (int e = 0; e < kChunk; ++e) a = fmaf(dy[e] * w[e], h[e], a);
  return a;
}

template <typename T, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_grad_kernel(const NormGradParams p) {
  __shared__ float slot[2][kMaxWarps];
  float w[NV][kChunk], acc[NV][kChunk];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x);
    Chunk8<T> c;
    c.load(static_cast<const T*>(p.w) + col, p.cols - col, p.vec != 0);
    c.get(w[j]);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) acc[j][e] = 0.0f;
  }
  GradRow<T, NV> cur, nxt;
  int64_t row = blockIdx.x;
  if (row < p.rows) cur.load(p, row);
  for (int it = 0; row < p.rows; row += gridDim.x, ++it) {
    const int64_t next = row + gridDim.x;
    if (next < p.rows) nxt.load(p, next);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) dot += grad_dot<T>(cur.dy[j], cur.h[j], w[j]);
    dot = cta_sum(dot, slot[it & 1]);  // two slots: a row's sums are read before the row after next writes
    const float rstd = cur.rstd;
    const float c = rstd * rstd * (dot / (float)p.cols);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      grad_chunk<T>(p, row, kChunk * (j * (int)blockDim.x + (int)threadIdx.x), cur.dy[j], cur.h[j], cur.dh[j], w[j],
                    rstd, c, acc[j]);
    cur = nxt;
  }
  if (p.partial) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x);
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col + e < p.cols) p.partial[(int64_t)blockIdx.x * p.cols + col + e] = acc[j][e];
    }
  }
}

// Rows too long for registers: dw in shared memory (each thread only ever touches its own
// columns), dy and h read again for dx.
template <typename T>
__global__ void __launch_bounds__(1024) rmsnorm_grad_wide_kernel(const NormGradParams p) {
  extern __shared__ float acc_s[];
  __shared__ float slot[2][kMaxWarps];
  const int step = kChunk * (int)blockDim.x;
  const int col0 = kChunk * (int)threadIdx.x;
  for (int col = col0; col < p.cols; col += step)
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (col + e < p.cols) acc_s[col + e] = 0.0f;
  int it = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
    Chunk8<T> cdy, ch, cdh, cw;
    float w[kChunk], dot = 0.0f;
    const auto load = [&](int col, bool with_dh) {
      const int left = p.cols - col;
      cdy.load(static_cast<const T*>(p.dy) + row * p.lddy + col, left, p.vec != 0);
      ch.load(static_cast<const T*>(p.h) + row * p.ldh + col, left, p.vec != 0);
      cw.load(static_cast<const T*>(p.w) + col, left, p.vec != 0);
      if (with_dh) cdh.load(static_cast<const T*>(p.dh) + row * p.lddh + col, left, p.vec != 0);
      cw.get(w);
    };
    for (int col = col0; col < p.cols; col += step) {
      load(col, false);
      dot += grad_dot<T>(cdy, ch, w);
    }
    dot = cta_sum(dot, slot[it & 1]);
    const float rstd = p.rstd[row];
    const float c = rstd * rstd * (dot / (float)p.cols);
    for (int col = col0; col < p.cols; col += step) {
      load(col, p.dh != nullptr);
      float acc[kChunk];
#pragma unroll
      for (int e = 0; e < kChunk; ++e) acc[e] = 0.0f;
      grad_chunk<T>(p, row, col, cdy, ch, cdh, w, rstd, c, acc);
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col + e < p.cols) acc_s[col + e] += acc[e];
    }
  }
  if (p.partial)
    for (int col = col0; col < p.cols; col += step)
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col + e < p.cols) p.partial[(int64_t)blockIdx.x * p.cols + col + e] = acc_s[col + e];
}

// dw = the CTAs' sums in CTA order: 32 columns per CTA, warp i adds a fixed share of the rows of
// `partial`, then the 32 warps' sums are added in warp order.
__global__ void __launch_bounds__(1024) grad_reduce_kernel(const float* __restrict__ partial, int n, int cols,
                                                           float* __restrict__ dw) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (int)blockIdx.x * 32 + lane;
  const int each = (n + 31) / 32;
  float a = 0.0f;
  if (col < cols)
    for (int i = warp * each; i < min(n, (warp + 1) * each); ++i) a += partial[(int64_t)i * cols + col];
  part[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && col < cols) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][lane];
    dw[col] = s;
  }
}

// Shape of the gradient kernel: threads and chunks per thread that cover a row, 0 chunks for the
// wide form.  One chunk up to 4096 columns (512 threads), two up to 8192.
struct GradShape {
  int threads, chunks, ctas_per_sm;
};
GradShape grad_shape(int cols) {
  const int chunks = (cols + kChunk - 1) / kChunk;
  if (chunks <= 512) return {(chunks + 31) / 32 * 32, 1, std::max(1, 1024 / ((chunks + 31) / 32 * 32))};
  if (chunks <= 1024) return {(chunks + 63) / 64 * 32, 2, 1};
  return {1024, 0, 1};
}

template <typename T>
cudaError_t launch_backward(const NormGradParams& p, int grid, cudaStream_t stream) {
  const GradShape s = grad_shape(p.cols);
  if (s.chunks == 1) rmsnorm_grad_kernel<T, 1, 512><<<grid, s.threads, 0, stream>>>(p);
  else if (s.chunks == 2) rmsnorm_grad_kernel<T, 2, 512><<<grid, s.threads, 0, stream>>>(p);
  else rmsnorm_grad_wide_kernel<T><<<grid, s.threads, (size_t)p.cols * 4, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.partial) {
    grad_reduce_kernel<<<(p.cols + 31) / 32, 1024, 0, stream>>>(p.partial, grid, p.cols, p.dw);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace
}  // namespace f8

cudaError_t prepare_fp8_norm() {
  cudaError_t e = cudaFuncSetAttribute(f8::rmsnorm_grad_wide_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kNormGradMaxCols * 4);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(f8::rmsnorm_grad_wide_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kNormGradMaxCols * 4);
  return e;
}

cudaError_t launch_fp8_rmsnorm(int type, const NormParams& p, cudaStream_t stream) {
  return type == SGEMM_BF16 ? f8::launch_forward<__nv_bfloat16>(p, stream) : f8::launch_forward<float>(p, stream);
}

int fp8_rmsnorm_backward_grid(int, int64_t rows, int cols, int sm_count) {
  return (int)std::min<int64_t>(rows, (int64_t)sm_count * f8::grad_shape(cols).ctas_per_sm);
}

cudaError_t launch_fp8_rmsnorm_backward(int type, const NormGradParams& p, int grid, cudaStream_t stream) {
  return type == SGEMM_BF16 ? f8::launch_backward<__nv_bfloat16>(p, grid, stream)
                            : f8::launch_backward<float>(p, grid, stream);
}

}  // namespace sgemm_impl
