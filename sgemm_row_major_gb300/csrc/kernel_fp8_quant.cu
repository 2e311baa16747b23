// kernel_fp8_quant.cu -- 8-bit codes and scales of an FP32 or BF16 matrix in groups of 1 x 128,
// 128 x 1 or 128 x 128 elements.
//
//     s = max(amax / top, 2^-126),   code = rn8(x * rn(1 / s))
//
// One CTA takes a 128 x 128 tile whatever the groups: its 256 threads load the whole tile as
// 16-byte chunks before they use any (64 KB of FP32 or 32 KB of BF16 in flight per CTA), keep it in
// registers, find the groups' largest values -- across the lanes of a row (1 x 128), down the
// thread's own columns and then across the warps through shared memory (128 x 1, 128 x 128) -- and
// write the codes of their own elements.  So X is read once and the pass is an HBM stream: FP32 4096 x
// 4096 in 128 x 128 groups 15.4 us (5.5 TB/s of 6.8 measured for a copy), BF16 16384 x 4096 in 128 x 1
// or 1 x 128 groups 38 us (5.3 TB/s), FP32 8192 x 4096 28 us (5.9 TB/s); what is missing is the start and the end,
// when not all SMs load.  Rows that do not begin at multiples of 16 bytes: BF16 8192 x 4095 26 to 32 us.
#include "fp8_common.cuh"
#include "fp8_internal.h"

namespace sgemm_impl {
namespace f8 {
namespace {

constexpr int kTile = 128;
constexpr int kQuantThreads = 256;
enum Groups { kRow = 0, kCol = 1, kBlock = 2 };

template <typename T>
constexpr int kCtas = sizeof(T) == 2 ? 3 : 2;  // per SM: 128 KB of FP32 or 96 KB of BF16 in flight

// What the threads of a CTA share of a tile: its place, and (128 x 1, 128 x 128) the partial maxima.
// VEC: rows of X start at multiples of 16 bytes and hold whole chunks of V elements.
template <typename T, int G, bool VEC>
struct Quant {
  static constexpr int V = Chunk<T>::V;
  static constexpr int kLanesPerRow = kTile / V;                     // 32 (FP32) or 16 (BF16)
  static constexpr int kRowsPerPass = kQuantThreads / kLanesPerRow;  // 8 or 16
  static constexpr int kPasses = kTile / kRowsPerPass;

  // Scales and codes of the tile.  CHECK = false: an infinite x is not expected; returns true when a
  // group of this thread's has one (that group is then to be done again with CHECK).
  template <bool CHECK>
  static __device__ __forceinline__ bool tile(const QuantParams& p, int64_t rt, int ct, float (*part)[kTile]) {
    const int lr = (int)threadIdx.x / kLanesPerRow, lc = (int)threadIdx.x % kLanesPerRow;
    const int rows = (int)min((int64_t)kTile, p.rows - rt * kTile) - lr;  // of the tile, from this thread's first
    const int64_t col = (int64_t)ct * kTile + lc * V;
    const int left = (int)max((int64_t)0, min((int64_t)V, p.cols - col));  // elements of its chunks
    const bool e5m2 = p.format == SGEMM_FP8_E5M2;
    const float top = e5m2 ? kMaxE5M2 : kMaxE4M3;
    const auto mag = [](float x) { return CHECK ? finite_abs(x) : fabsf(x); };  // fmaxf passes over a NaN
    Chunk<T> c[kPasses];
    {
      const T* x = static_cast<const T*>(p.x) + (rt * kTile + lr) * p.ldx + col;
      const Rows<T> all(p.x, p.rows, p.ldx, p.cols, p.guard);
      constexpr int kBatch = VEC ? kPasses : 4;  // chunks on their way at once
#pragma unroll
      for (int i0 = 0; i0 < kPasses; i0 += kBatch) {
        Loading<T, VEC> l[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i, x += kRowsPerPass * p.ldx)
          l[i].load(x, (i0 + i) * kRowsPerPass < rows ? left : 0, all);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) c[i0 + i] = l[i].get();
      }
    }
    const int64_t scales = extent(G == kRow ? p.rows : (p.rows + kTile - 1) / kTile, p.lds, G == kCol ? p.cols : (p.cols + kTile - 1) / kTile);
    bool again = false;
    float inv[G == kCol ? V : 1];
    if constexpr (G != kRow) {
      float m[G == kCol ? V : 1];
#pragma unroll
      for (int e = 0; e < (G == kCol ? V : 1); ++e) m[e] = 0.0f;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        float v[V];
        c[i].get(v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float& x = m[G == kCol ? e : 0];
          x = fmaxf(x, mag(v[e]));
        }
      }
      if constexpr (G == kBlock) {
        const float w = lanes_max<32>(m[0]);
        if ((threadIdx.x & 31) == 0) part[0][threadIdx.x >> 5] = w;
        __syncthreads();
        float a = part[0][0];
#pragma unroll
        for (int i = 1; i < kQuantThreads / 32; ++i) a = fmaxf(a, part[0][i]);
        again = !CHECK && a > kMaxFloat;
        const float s = group_scale(a, top);
        if (threadIdx.x == 0) put_at(p.guard, kSiteScale, p.s, rt * p.lds + ct, scales, s);
        inv[0] = __frcp_rn(s);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) part[lr][lc * V + e] = m[e];
        __syncthreads();
        if (threadIdx.x < kTile) {
          float a = 0.0f;
#pragma unroll
          for (int i = 0; i < kRowsPerPass; ++i) a = fmaxf(a, part[i][threadIdx.x]);
          const float s = group_scale(a, top);
          part[0][threadIdx.x] = s;
          const int64_t at = (int64_t)ct * kTile + threadIdx.x;
          if (at < p.cols) put_at(p.guard, kSiteScale, p.s, rt * p.lds + at, scales, s);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float s = part[0][lc * V + e];
          again = again || (!CHECK && s > kMaxFloat);
          inv[e] = __frcp_rn(s);
        }
      }
    }
    uint8_t* q = p.q + (rt * kTile + lr) * p.ldq + col;
    const Rows<uint8_t> codes(p.q, p.rows, p.ldq, p.cols, p.guard);
#pragma unroll
    for (int i = 0; i < kPasses; ++i, q += kRowsPerPass * p.ldq) {
      const bool in = i * kRowsPerPass < rows;
      float v[V];
      c[i].get(v);
      if (G == kRow) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) m = fmaxf(m, mag(v[e]));
        m = lanes_max<kLanesPerRow>(m);
        again = again || (!CHECK && m > kMaxFloat);
        const float s = group_scale(m, top);
        inv[0] = __frcp_rn(s);
        if (lc == 0 && in) put_at(p.guard, kSiteScale, p.s, (rt * kTile + lr + i * kRowsPerPass) * p.lds + ct, scales, s);
      }
      if (in) {
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = inv[G == kCol ? e : 0];
        store_codes<V, CHECK>(q, v, f, left, e5m2, codes);
      }
    }
    return again;
  }

  static __device__ __noinline__ void checked_tile(const QuantParams& p, int64_t rt, int ct, float (*part)[kTile]) {
    tile<true>(p, rt, ct, part);
  }
};

template <typename T, int G, bool VEC>
__global__ void __launch_bounds__(kQuantThreads, kCtas<T>) quantize_kernel(const __grid_constant__ QuantParams p,
                                                                           int col_tiles) {
  using Q = Quant<T, G, VEC>;
  __shared__ float part[G == kCol ? Q::kRowsPerPass : 1][kTile];
  const int64_t rt = (int64_t)blockIdx.x / col_tiles;
  const int ct = (int)(blockIdx.x - rt * col_tiles);
  // the tests for infinities cost as much as everything else here: a tile that has one is done again
  if (__syncthreads_or(Q::template tile<false>(p, rt, ct, part))) Q::checked_tile(p, rt, ct, part);
}

template <typename T>
cudaError_t launch(int block_rows, int block_cols, const QuantParams& p, cudaStream_t stream) {
  const int64_t ct = (p.cols + kTile - 1) / kTile, rt = (p.rows + kTile - 1) / kTile;
  const dim3 grid((unsigned)(ct * rt));
  const auto run = [&](auto kernel) { kernel<<<grid, kQuantThreads, 0, stream>>>(p, (int)ct); };
  const bool vec = p.x_vec && p.cols % Chunk<T>::V == 0;
  if (block_rows == 1) vec ? run(quantize_kernel<T, kRow, true>) : run(quantize_kernel<T, kRow, false>);
  else if (block_cols == 1) vec ? run(quantize_kernel<T, kCol, true>) : run(quantize_kernel<T, kCol, false>);
  else vec ? run(quantize_kernel<T, kBlock, true>) : run(quantize_kernel<T, kBlock, false>);
  return cudaGetLastError();
}

}  // namespace
}  // namespace f8

cudaError_t launch_fp8_quantize(int type, int block_rows, int block_cols, const QuantParams& p, cudaStream_t stream) {
  return type == SGEMM_BF16 ? f8::launch<__nv_bfloat16>(block_rows, block_cols, p, stream)
                            : f8::launch<float>(block_rows, block_cols, p, stream);
}

}  // namespace sgemm_impl
