// kernel_fp8_norm.cu -- RMS norm with residual addition and 8-bit output, and its gradients.
//
// Forward, for a row of n columns:   h = x + r,  rstd = (sum h^2 / n + eps)^(-1/2),  y = h rstd w,
// and y in E4M3 codes with a scale per 128 columns.  One CTA per row: a thread keeps its 8-column
// chunks of h in registers between the sum and the output, so x and r are read once and h and the
// codes written once (an HBM stream: 7 bytes per element of a BF16 row with a residual).  16
// neighbouring threads hold one group of 128 columns, so a group's largest value is a shuffle away.
// BF16 16384 x 4096 with a residual: 80 us, 5.9 TB/s of 6.8 measured for a copy (FP32 8192 x 4096 68 us,
// 6.4 TB/s); one row of 4096: 3.1 us, which is a launch and one memory latency.  Rows that begin anywhere
// take more instructions per byte (fp8_common.cuh, Loading): 8192 x 4095 BF16 66 us, 3.6 TB/s, FP32 112 us.
//
// Backward:   dx = rstd (dy w - h rstd^2 mean(dy w h)) + dh,   dw = sum_rows dy h rstd.
// A persistent grid: a CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ..., its threads own
// fixed columns and keep their part of dw in registers (the wide form: in shared memory), so dw
// costs no traffic per row; the CTAs' sums go to `partial` and a second kernel adds them in CTA
// order.  Rows that begin at multiples of 16 bytes are copied to a ring in shared memory by bulk copies
// several rows ahead (192 KB in flight per SM), others are loaded one row ahead into registers.
// BF16 8192 x 4096 with dh: 50 us, 5.4 TB/s (62 us with loads one row ahead); the second kernel and the
// first rows' latency are about 5 us of it.  8192 x 4095, one row ahead: BF16 89 us, FP32 119 us.
#include <algorithm>

#include "fp8_common.cuh"
#include "fp8_internal.h"

namespace sgemm_impl {
namespace f8 {
namespace {

constexpr int kChunk = 8;         // columns a thread takes at a time
constexpr int kMaxWarps = 32;

// 8 columns: one 16-byte vector of BF16, two of FP32; load() sends for them, get() waits for them.
template <typename T, bool VEC>
struct Chunk8 {
  static constexpr int kVecs = kChunk / Chunk<T>::V;
  Loading<T, VEC> c[kVecs];
  __device__ __forceinline__ void load(const T* p, int n, const Rows<T>& m) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) c[i].load(p + i * Chunk<T>::V, (int64_t)(n - i * Chunk<T>::V), m);
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) c[i].get().get(v + i * Chunk<T>::V);
  }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const float* v, int n, const Rows<T>& m) {
#pragma unroll
  for (int i = 0; i < kChunk / Chunk<T>::V; ++i)
    store_chunk<T, VEC>(p + i * Chunk<T>::V, v + i * Chunk<T>::V, (int64_t)(n - i * Chunk<T>::V), m);
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
template <typename T, bool VEC>
__device__ __forceinline__ void emit(const NormParams& p, int64_t row, int col, const float* h, float rstd) {
  const int left = p.cols - col;
  float y[kChunk];
  {
    Chunk8<T, VEC> w;
    w.load(static_cast<const T*>(p.w) + col, left, Rows<T>(p.w, 1, 0, p.cols, p.guard));
    w.get(y);
  }
#pragma unroll
  for (int e = 0; e < kChunk; ++e) y[e] = h[e] * rstd * y[e];  // columns past the end: h = 0
  if (p.y && left > 0)
    store8<T, VEC>(static_cast<T*>(p.y) + row * p.ldy + col, y, left, Rows<T>(p.y, p.rows, p.ldy, p.cols, p.guard));
  if (p.q) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) m = fmaxf(m, finite_abs(y[e]));
    const float s = group_scale(lanes_max<16>(m), kMaxE4M3);
    if (left > 0) {
      if (col % 128 == 0)
        put_at(p.guard, kSiteScale, p.s, row * p.lds + col / 128, extent(p.rows, p.lds, (p.cols - 1) / 128 + 1), s);
      float inv[kChunk];
#pragma unroll
      for (int e = 0; e < kChunk; ++e) inv[e] = __frcp_rn(s);
      store_codes<kChunk, true>(p.q + row * p.ldq + col, y, inv, left, false,
                                Rows<uint8_t>(p.q, p.rows, p.ldq, p.cols, p.guard));
    }
  }
}

// A chunk of x and of r, whose sum is h.
template <typename T, bool VEC>
struct Sum8 {
  Chunk8<T, VEC> x, r;
  __device__ __forceinline__ void load(const NormParams& p, int64_t row, int col) {
    const int left = p.cols - col;
    x.load(static_cast<const T*>(p.x) + row * p.ldx + col, left, Rows<T>(p.x, p.rows, p.ldx, p.cols, p.guard));
    if (p.r) r.load(static_cast<const T*>(p.r) + row * p.ldr + col, left, Rows<T>(p.r, p.rows, p.ldr, p.cols, p.guard));
  }
  __device__ __forceinline__ void get(const NormParams& p, float* h) const {
    x.get(h);
    if (p.r) {
      float b[kChunk];
      r.get(b);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) h[e] += b[e];
    }
  }
};

// NV chunks per thread; chunk j of thread t is columns 8 (j blockDim.x + t) .. + 7.
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slot[kMaxWarps];
  const int64_t row = blockIdx.x;
  float h[NV][kChunk];
  float ss = 0.0f;
  if (VEC) {  // (the compiler sends for all of them first)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Sum8<T, VEC> in;
      in.load(p, row, kChunk * (j * (int)blockDim.x + (int)threadIdx.x));
      in.get(p, h[j]);
    }
  } else {
    Sum8<T, VEC> in[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) in[j].load(p, row, kChunk * (j * (int)blockDim.x + (int)threadIdx.x));
#pragma unroll
    for (int j = 0; j < NV; ++j) in[j].get(p, h[j]);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) a = fmaf(h[j][e], h[j][e], a);
    ss += a;
  }
  const float rstd = __frsqrt_rn(cta_sum(ss, slot) / (float)p.cols + p.eps);
  if (p.rstd && threadIdx.x == 0) put_at(p.guard, kSiteRowStat, p.rstd, row, p.rows, rstd);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x);
    if (p.h && col < p.cols)
      store8<T, VEC>(static_cast<T*>(p.h) + row * p.ldh + col, h[j], p.cols - col, Rows<T>(p.h, p.rows, p.ldh, p.cols, p.guard));
    emit<T, VEC>(p, row, col, h[j], rstd);
  }
}

// Rows too long for registers: a second pass reads x and r again (from L2) for the output.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) rmsnorm_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slot[kMaxWarps];
  const int64_t row = blockIdx.x;
  const int step = kChunk * (int)blockDim.x;
  float ss = 0.0f;
  for (int64_t c0 = 0; c0 < p.cols; c0 += step) {  // 64-bit: c0 + step may pass 2^31
    float h[kChunk];
    const int64_t col = c0 + kChunk * (int)threadIdx.x;
    if (col >= p.cols) continue;
    Sum8<T, VEC> in;
    in.load(p, row, (int)col);
    in.get(p, h);
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) a = fmaf(h[e], h[e], a);
    ss += a;
  }
  const float rstd = __frsqrt_rn(cta_sum(ss, slot) / (float)p.cols + p.eps);
  if (p.rstd && threadIdx.x == 0) put_at(p.guard, kSiteRowStat, p.rstd, row, p.rows, rstd);
  for (int64_t c0 = 0; c0 < p.cols; c0 += step) {
    float h[kChunk];
    // every lane stays in the loop (the groups' shuffles); past the end it works on no columns
    const int col = (int)min(c0 + kChunk * (int)threadIdx.x, ((int64_t)p.cols + 7) / 8 * 8);
    Sum8<T, VEC> in;
    in.load(p, row, col);
    in.get(p, h);
    // h may overwrite x or r: only this thread reads these columns, and it has
    if (p.h && col < p.cols)
      store8<T, VEC>(static_cast<T*>(p.h) + row * p.ldh + col, h, p.cols - col, Rows<T>(p.h, p.rows, p.ldh, p.cols, p.guard));
    emit<T, VEC>(p, row, col, h, rstd);
  }
}

constexpr int kRegCols = 32768;  // 1024 threads x 4 chunks

template <typename T, bool VEC>
cudaError_t launch_forward(const NormParams& p, cudaStream_t stream) {
  const int chunks = (int)(((int64_t)p.cols + kChunk - 1) / kChunk);
  const dim3 grid((unsigned)p.rows);
  // One chunk per thread up to 1024 columns, two up to 8192, then four: more chunks per thread keep more bytes
  // in flight, more threads finish a row sooner.  Measured with 1, 2 and 4 chunks, us for 48 M BF16 elements
  // (and for one row): 1024 columns 69, 56, 54 (2.2, 2.6, 3.6); 4096 76, 58, 55 (2.6, 2.9, 3.8); 8192 88, 67, 58
  // (3.2, 3.3, 4.2); 16384 with 2 and 4 81, 61 (4.1, 4.8); FP32 within 2% up to 4096 columns.  At 32768
  // columns the wide form takes 76 us, four chunks 71.
  const auto threads = [&](int nv) { return std::min(1024, (chunks + 32 * nv - 1) / (32 * nv) * 32); };
  if (p.cols > kRegCols) rmsnorm_wide_kernel<T, VEC><<<grid, 1024, 0, stream>>>(p);
  else if (chunks <= 128) rmsnorm_kernel<T, 1, VEC><<<grid, threads(1), 0, stream>>>(p);
  else if (chunks <= 1024) rmsnorm_kernel<T, 2, VEC><<<grid, threads(2), 0, stream>>>(p);
  else rmsnorm_kernel<T, 4, VEC><<<grid, threads(4), 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ backward

// A column of this CTA's sums of dW.
__device__ __forceinline__ void put_partial(const NormGradParams& p, int col, float v) {
  put_at(p.guard, kSitePart, p.partial, (int64_t)blockIdx.x * p.cols + col, (int64_t)gridDim.x * p.cols, v);
}

template <typename T, int NV, bool VEC>
struct GradRow {  // a thread's chunks of dy, h and dh of one row
  Chunk8<T, VEC> dy[NV], h[NV], dh[NV];
  float rstd;
  __device__ __forceinline__ void load(const NormGradParams& p, int64_t row) {
    rstd = get_at(p.guard, kSiteRowStat, p.rstd, row, p.rows);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x), left = p.cols - col;
      dy[j].load(static_cast<const T*>(p.dy) + row * p.lddy + col, left, Rows<T>(p.dy, p.rows, p.lddy, p.cols, p.guard));
      h[j].load(static_cast<const T*>(p.h) + row * p.ldh + col, left, Rows<T>(p.h, p.rows, p.ldh, p.cols, p.guard));
      if (p.dh)
        dh[j].load(static_cast<const T*>(p.dh) + row * p.lddh + col, left,
                                 Rows<T>(p.dh, p.rows, p.lddh, p.cols, p.guard));
    }
  }
};

// One chunk of dx, and its part of dw added to acc.
template <typename T, bool VEC>
__device__ __forceinline__ void grad_chunk(const NormGradParams& p, int64_t row, int col, const Chunk8<T, VEC>& cdy,
                                           const Chunk8<T, VEC>& ch, const Chunk8<T, VEC>& cdh, const float* w, float rstd,
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
  if (col < p.cols)
    store8<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx + col, dx, p.cols - col, Rows<T>(p.dx, p.rows, p.lddx, p.cols, p.guard));
}

template <typename T, bool VEC>
__device__ __forceinline__ float grad_dot(const Chunk8<T, VEC>& cdy, const Chunk8<T, VEC>& ch, const float* w) {
  float dy[kChunk], h[kChunk], a = 0.0f;
  cdy.get(dy);
  ch.get(h);
#pragma unroll
  for (int e = 0; e < kChunk; ++e) a = fmaf(dy[e] * w[e], h[e], a);
  return a;
}

template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(512) rmsnorm_grad_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ float slot[2][kMaxWarps];
  float w[NV][kChunk], acc[NV][kChunk];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x);
    Chunk8<T, VEC> c;
    c.load(static_cast<const T*>(p.w) + col, p.cols - col, Rows<T>(p.w, 1, 0, p.cols, p.guard));
    c.get(w[j]);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) acc[j][e] = 0.0f;
  }
  GradRow<T, NV, VEC> cur, nxt;
  int64_t row = blockIdx.x;
  if (row < p.rows) cur.load(p, row);
  for (int it = 0; row < p.rows; row += gridDim.x, ++it) {
    const int64_t next = row + gridDim.x;
    if (next < p.rows) nxt.load(p, next);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) dot += grad_dot<T, VEC>(cur.dy[j], cur.h[j], w[j]);
    dot = cta_sum(dot, slot[it & 1]);  // two slots: a row's sums are read before the row after next writes
    const float rstd = cur.rstd;
    const float c = rstd * rstd * (dot / (float)p.cols);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      grad_chunk<T, VEC>(p, row, kChunk * (j * (int)blockDim.x + (int)threadIdx.x), cur.dy[j], cur.h[j], cur.dh[j], w[j],
                    rstd, c, acc[j]);
    cur = nxt;
  }
  if (p.partial) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x);
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col + e < p.cols) put_partial(p, col + e, acc[j][e]);
    }
  }
}

// The same with the rows' copies in a ring of `depth` slots of {dy, h, dh} in shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
constexpr int kMaxDepth = 16;

template <typename T, int NV>
__global__ void __launch_bounds__(512, 1) rmsnorm_grad_ring_kernel(const __grid_constant__ NormGradParams p, int depth) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kMaxDepth];
  __shared__ float slot[2][kMaxWarps];
  const uint32_t row_bytes = (uint32_t)p.cols * sizeof(T), parts = p.dh ? 3 : 2;  // a multiple of 16
  const uint32_t slot_bytes = 3 * row_bytes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const auto load = [&](int s, int64_t row) {  // one thread
    const uint32_t bar = smem_addr(&full[s]), dst = smem_addr(ring) + (uint32_t)s * slot_bytes;
    mbar_arrive_expect_tx(bar, parts * row_bytes);
    const auto part = [&](int i, const void* base, int64_t ld) {
      const T* src = static_cast<const T*>(base) + row * ld;
      if (Rows<T>(base, p.rows, ld, p.cols, p.guard).holds(kSiteIn, src, p.cols)) bulk_load(dst + i * row_bytes, src, row_bytes, bar);
    };
    part(0, p.dy, p.lddy);
    part(1, p.h, p.ldh);
    if (p.dh) part(2, p.dh, p.lddh);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < depth; ++s) mbar_init(smem_addr(&full[s]), 1);
    fence_mbar_init();
    for (int s = 0; s < depth; ++s)
      if (blockIdx.x + (int64_t)s * gridDim.x < p.rows) load(s, blockIdx.x + (int64_t)s * gridDim.x);
  }
  float w[NV][kChunk], acc[NV][kChunk];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x);
    Chunk8<T, true> c;
    c.load(static_cast<const T*>(p.w) + col, p.cols - col, Rows<T>(p.w, 1, 0, p.cols, p.guard));
    c.get(w[j]);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) acc[j][e] = 0.0f;
  }
  __syncthreads();
  int s = 0;
  uint32_t lap = 0;
  bool ok = true;  // the same in every thread: each waits for the same phases
  int it = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
    const float rstd = get_at(p.guard, kSiteRowStat, p.rstd, row, p.rows);
    ok = ok && mbar_wait(smem_addr(&full[s]), lap & 1u, p.timeout_ns);
    if (!ok && threadIdx.x == 0) atomicOr(p.fault, (unsigned)kFaultFullWait);
    const T* base = reinterpret_cast<const T*>(ring + (size_t)s * slot_bytes);
    Chunk8<T, true> dy[NV], h[NV], dh[NV];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x), left = p.cols - col;
      const Rows<T> in(base, 1, 0, 3 * p.cols, p.guard);
      dy[j].load(base + col, left, in);
      h[j].load(base + p.cols + col, left, in);
      if (p.dh) dh[j].load(base + 2 * p.cols + col, left, in);
      dot += grad_dot<T, true>(dy[j], h[j], w[j]);
    }
    dot = cta_sum(dot, slot[it & 1]);  // its barrier: every thread has read the row
    if (threadIdx.x == 0 && ok && row + (int64_t)depth * gridDim.x < p.rows) load(s, row + (int64_t)depth * gridDim.x);
    const float c = rstd * rstd * (dot / (float)p.cols);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      grad_chunk<T, true>(p, row, kChunk * (j * (int)blockDim.x + (int)threadIdx.x), dy[j], h[j], dh[j], w[j], rstd, c, acc[j]);
    if (++s == depth) {
      s = 0;
      ++lap;
    }
  }
  if (p.partial) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = kChunk * (j * (int)blockDim.x + (int)threadIdx.x);
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col + e < p.cols) put_partial(p, col + e, acc[j][e]);
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
    Chunk8<T, false> cdy, ch, cdh, cw;
    float w[kChunk], dot = 0.0f;
    const auto load = [&](int col, bool with_dh) {
      const int left = p.cols - col;
      cdy.load(static_cast<const T*>(p.dy) + row * p.lddy + col, left, Rows<T>(p.dy, p.rows, p.lddy, p.cols, p.guard));
      ch.load(static_cast<const T*>(p.h) + row * p.ldh + col, left, Rows<T>(p.h, p.rows, p.ldh, p.cols, p.guard));
      cw.load(static_cast<const T*>(p.w) + col, left, Rows<T>(p.w, 1, 0, p.cols, p.guard));
      if (with_dh)
        cdh.load(static_cast<const T*>(p.dh) + row * p.lddh + col, left,
                                 Rows<T>(p.dh, p.rows, p.lddh, p.cols, p.guard));
      cw.get(w);
    };
    for (int col = col0; col < p.cols; col += step) {
      load(col, false);
      dot += grad_dot<T, false>(cdy, ch, w);
    }
    dot = cta_sum(dot, slot[it & 1]);
    const float rstd = get_at(p.guard, kSiteRowStat, p.rstd, row, p.rows);
    const float c = rstd * rstd * (dot / (float)p.cols);
    for (int col = col0; col < p.cols; col += step) {
      load(col, p.dh != nullptr);
      float acc[kChunk];
#pragma unroll
      for (int e = 0; e < kChunk; ++e) acc[e] = 0.0f;
      grad_chunk<T, false>(p, row, col, cdy, ch, cdh, w, rstd, c, acc);
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col + e < p.cols) acc_s[col + e] += acc[e];
    }
  }
  if (p.partial)
    for (int col = col0; col < p.cols; col += step)
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col + e < p.cols) put_partial(p, col + e, acc_s[col + e]);
}

// dw = the CTAs' sums in CTA order: 32 columns per CTA, warp i adds a fixed share of the rows of
// `partial`, then the 32 warps' sums are added in warp order.
__global__ void __launch_bounds__(1024) grad_reduce_kernel(const float* __restrict__ partial, int n, int cols,
                                                           float* __restrict__ dw, const Guard guard) {
  __shared__ float part[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // a programmatic dependent of the kernel above
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (int)blockIdx.x * 32 + lane;
  const int each = (n + 31) / 32;
  float a = 0.0f;
  if (col < cols)
    for (int i = warp * each; i < min(n, (warp + 1) * each); ++i) a += get_at(guard, kSitePart, partial, (int64_t)i * cols + col, (int64_t)n * cols);
  part[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && col < cols) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][lane];
    put_at(guard, kSiteOut, dw, col, cols, s);
  }
}

// Shape of the gradient kernel: threads and chunks per thread that cover a row (0 chunks: the wide
// form), and the ring's slots (0: no ring).  With a ring of BF16 rows two chunks beyond 2048 columns,
// so that two CTAs per SM take turns at their rows' sums (8192 x 4096: 49 us, with one CTA of 512
// threads 55 us; in FP32 93 against 86 us; but 300 rows of 4096 11.3 us, with one chunk 8.4).  The ring
// from 512 columns on, us with and without it for 48 M BF16 elements: 128 columns 121, 118; 256 69, 74; 512
// 66, 73; 2048 65, 74; FP32 at 512 93, 100.
struct GradShape {
  int threads, chunks, ctas_per_sm, depth;
};
constexpr int kRingBytes = 192 * 1024;
GradShape grad_shape(int type, int cols, bool vec) {
  const int chunks = (cols + kChunk - 1) / kChunk, row = 3 * cols * (type == SGEMM_BF16 ? 2 : 4);
  if (chunks > 1024) return {1024, 0, 1, 0};
  const bool whole = vec && chunks >= 64;
  const int per_thread = chunks <= (whole && type == SGEMM_BF16 ? 256 : 512) ? 1 : 2;
  const int threads = (chunks + 32 * per_thread - 1) / (32 * per_thread) * 32;
  if (whole) {
    const int ctas = std::max(1, 512 / threads);
    return {threads, per_thread, ctas, std::min(kMaxDepth, kRingBytes / ctas / row)};
  }
  return {threads, per_thread, std::max(1, 512 / threads), 0};
}

template <typename T>
cudaError_t launch_backward(int type, const NormGradParams& p, int grid, cudaStream_t stream) {
  const GradShape s = grad_shape(type, p.cols, p.vec != 0);
  const size_t ring = (size_t)s.depth * 3 * p.cols * sizeof(T);
  if (s.depth >= 2 && s.chunks == 1) rmsnorm_grad_ring_kernel<T, 1><<<grid, s.threads, ring, stream>>>(p, s.depth);
  else if (s.depth >= 2) rmsnorm_grad_ring_kernel<T, 2><<<grid, s.threads, ring, stream>>>(p, s.depth);
  else if (s.chunks == 1 && p.vec) rmsnorm_grad_kernel<T, 1, true><<<grid, s.threads, 0, stream>>>(p);
  else if (s.chunks == 1) rmsnorm_grad_kernel<T, 1, false><<<grid, s.threads, 0, stream>>>(p);
  else if (s.chunks == 2) rmsnorm_grad_kernel<T, 2, false><<<grid, s.threads, 0, stream>>>(p);
  else rmsnorm_grad_wide_kernel<T><<<grid, s.threads, (size_t)p.cols * 4, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.partial) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.cols + 31) / 32));
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const float* partial = p.partial;
    e = cudaLaunchKernelEx(&cfg, grad_reduce_kernel, partial, grid, p.cols, p.dw, p.guard);
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
  for (const void* kernel : {reinterpret_cast<const void*>(f8::rmsnorm_grad_ring_kernel<float, 1>),
                             reinterpret_cast<const void*>(f8::rmsnorm_grad_ring_kernel<float, 2>),
                             reinterpret_cast<const void*>(f8::rmsnorm_grad_ring_kernel<__nv_bfloat16, 1>),
                             reinterpret_cast<const void*>(f8::rmsnorm_grad_ring_kernel<__nv_bfloat16, 2>)})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, f8::kRingBytes);
  return e;
}

cudaError_t launch_fp8_rmsnorm(int type, const NormParams& p, cudaStream_t stream) {
  if (type == SGEMM_BF16)
    return p.vec ? f8::launch_forward<__nv_bfloat16, true>(p, stream) : f8::launch_forward<__nv_bfloat16, false>(p, stream);
  return p.vec ? f8::launch_forward<float, true>(p, stream) : f8::launch_forward<float, false>(p, stream);
}

int fp8_rmsnorm_backward_grid(int type, int64_t rows, int cols, bool vec, int sm_count) {
  return (int)std::min<int64_t>(rows, (int64_t)sm_count * f8::grad_shape(type, cols, vec).ctas_per_sm);
}

cudaError_t launch_fp8_rmsnorm_backward(int type, const NormGradParams& p, int grid, cudaStream_t stream) {
  return type == SGEMM_BF16 ? f8::launch_backward<__nv_bfloat16>(type, p, grid, stream)
                            : f8::launch_backward<float>(type, p, grid, stream);
}

}  // namespace sgemm_impl
