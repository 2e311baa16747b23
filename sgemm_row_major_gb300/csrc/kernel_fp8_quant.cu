// kernel_fp8_quant.cu -- 8-bit codes and scales of an FP32 or BF16 matrix in groups of 1 x 128,
// 128 x 1 or 128 x 128 elements.
//
//     s = max(amax / top, 2^-126),   code = rn8(x * rn(1 / s))
//
// One CTA takes a 128 x 128 tile whatever the groups: its 256 threads load the whole tile as
// 16-byte chunks before they use any (64 KB of FP32 or 32 KB of BF16 in flight per CTA), keep it in
// registers, find the groups' largest values -- across the lanes of a row (1 x 128), down the
// thread's own columns and then across the warps through shared memory (128 x 1, 128 x 128) -- and
// write the codes of their own elements.  So X is read once and the pass is an HBM stream.
#include "fp8_common.cuh"
#include "fp8_internal.h"

namespace sgemm_impl {
namespace f8 {
namespace {

constexpr int kTile = 128;
constexpr int kQuantThreads = 256;
enum Groups { kRow = 0, kCol = 1, kBlock = 2 };

template <typename T, int G>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantParams p, int col_tiles) {
  constexpr int V = Chunk<T>::V;
  constexpr int kLanesPerRow = kTile / V;                      // 32 (FP32) or 16 (BF16)
  constexpr int kRowsPerPass = kQuantThreads / kLanesPerRow;   // 8 or 16
  constexpr int kPasses = kTile / kRowsPerPass;
  __shared__ float part[G == kRow ? 1 : kRowsPerPass][G == kRow ? 1 : kTile];

  const int64_t rt = (int64_t)blockIdx.x / col_tiles;
  const int ct = (int)(blockIdx.x - rt * col_tiles);
  const int lr = (int)threadIdx.x / kLanesPerRow, lc = (int)threadIdx.x % kLanesPerRow;
  const int64_t row0 = rt * kTile + lr, col = (int64_t)ct * kTile + lc * V;
  const int64_t left = p.cols - col;  // elements of this thread's chunk that exist (may be <= 0 or > V)
  const T* x = static_cast<const T*>(p.x) + row0 * p.ldx + col;
  const bool e5m2 = p.format == SGEMM_FP8_E5M2;
  const float top = e5m2 ? kMaxE5M2 : kMaxE4M3;

  Chunk<T> c[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const bool in = row0 + i * kRowsPerPass < p.rows;
    c[i] = load_chunk(x + (int64_t)i * kRowsPerPass * p.ldx, in ? left : 0, p.vec != 0);
  }

  float scale[V];  // of the thread's columns (128 x 1) or of everything (128 x 128: the first)
  if (G != kRow) {
    float m[V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      float v[V];
      c[i].get(v);
#pragma unroll
      for (int e = 0; e < V; ++e) m[e] = fmaxf(m[e], finite_abs(v[e]));
    }
#pragma unroll
    for (int e = 0; e < V; ++e) part[lr][lc * V + e] = m[e];
    __syncthreads();
    if (threadIdx.x < kTile) {
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < kRowsPerPass; ++i) a = fmaxf(a, part[i][threadIdx.x]);
      if (G == kBlock) a = lanes_max<32>(a);
      part[0][threadIdx.x] = a;
    }
    __syncthreads();
    if (G == kCol) {
#pragma unroll
      for (int e = 0; e < V; ++e) scale[e] = group_scale(part[0][lc * V + e], top);
      if (lr == 0)
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e < left) p.s[rt * p.lds + col + e] = scale[e];
    } else {
      scale[0] = group_scale(fmaxf(fmaxf(part[0][0], part[0][32]), fmaxf(part[0][64], part[0][96])), top);
      if (threadIdx.x == 0) p.s[rt * p.lds + ct] = scale[0];
    }
  }

  float inv[V];
  if (G == kCol) {
#pragma unroll
    for (int e = 0; e < V; ++e) inv[e] = __frcp_rn(scale[e]);
  } else if (G == kBlock) {
    inv[0] = __frcp_rn(scale[0]);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t row = row0 + i * kRowsPerPass;
    float v[V];
    c[i].get(v);
    if (G == kRow) {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) m = fmaxf(m, finite_abs(v[e]));
      const float s = group_scale(lanes_max<kLanesPerRow>(m), top);
      inv[0] = __frcp_rn(s);
      if (lc == 0 && row < p.rows) p.s[row * p.lds + ct] = s;
    }
    if (row < p.rows) {
      uint8_t* q = p.q + row * p.ldq + col;
      if (G == kCol) {
        float t[V];
#pragma unroll
        for (int e = 0; e < V; ++e) t[e] = v[e] * inv[e];
        store_codes<V>(q, t, 1.0f, left, p.vec != 0, e5m2);
      } else {
        store_codes<V>(q, v, inv[0], left, p.vec != 0, e5m2);
      }
    }
  }
}

template <typename T>
cudaError_t launch(int block_rows, int block_cols, const QuantParams& p, cudaStream_t stream) {
  const int64_t ct = (p.cols + kTile - 1) / kTile, rt = (p.rows + kTile - 1) / kTile;
  const dim3 grid((unsigned)(ct * rt));
  if (block_rows == 1) quantize_kernel<T, kRow><<<grid, kQuantThreads, 0, stream>>>(p, (int)ct);
  else if (block_cols == 1) quantize_kernel<T, kCol><<<grid, kQuantThreads, 0, stream>>>(p, (int)ct);
  else quantize_kernel<T, kBlock><<<grid, kQuantThreads, 0, stream>>>(p, (int)ct);
  return cudaGetLastError();
}

}  // namespace
}  // namespace f8

cudaError_t launch_fp8_quantize(int type, int block_rows, int block_cols, const QuantParams& p, cudaStream_t stream) {
  return type == SGEMM_BF16 ? f8::launch<__nv_bfloat16>(block_rows, block_cols, p, stream)
                            : f8::launch<float>(block_rows, block_cols, p, stream);
}

}  // namespace sgemm_impl
