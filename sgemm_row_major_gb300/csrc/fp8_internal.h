// fp8_internal.h -- host-side declarations of the 8-bit operators (sgemm_fp8.h).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "sgemm_fp8.h"

namespace sgemm_impl {

// What an entry point needs of the current device (set up by the first call on it; api.cu).
struct CallDevice {
  int sm_count = 0;
  int pair_clusters = 0;
  unsigned* fault = nullptr;
  cudaMemPool_t pool = nullptr;
};
int call_device(CallDevice* out);  // an sgemm_status

// ---- quantiser (kernel_fp8_quant.cu)
struct QuantParams {
  const void* x = nullptr;
  int64_t rows = 0, cols = 0, ldx = 0;
  uint8_t* q = nullptr;
  int64_t ldq = 0;
  float* s = nullptr;
  int64_t lds = 0;
  int format = 0;
  int vec = 0;  // 1: 16-byte loads and whole-vector stores are aligned
};
cudaError_t launch_fp8_quantize(int type, int block_rows, int block_cols, const QuantParams& p, cudaStream_t stream);

// ---- RMS norm (kernel_fp8_norm.cu)
struct NormParams {
  int64_t rows = 0;
  int cols = 0;
  const void *x = nullptr, *r = nullptr, *w = nullptr;
  int64_t ldx = 0, ldr = 0;
  float eps = 0.0f;
  void *h = nullptr, *y = nullptr;
  int64_t ldh = 0, ldy = 0;
  uint8_t* q = nullptr;
  int64_t ldq = 0;
  float *s = nullptr, *rstd = nullptr;
  int64_t lds = 0;
  int vec = 0;  // 1: every matrix row is aligned to its 8-element chunks
};
cudaError_t launch_fp8_rmsnorm(int type, const NormParams& p, cudaStream_t stream);

struct NormGradParams {
  int64_t rows = 0;
  int cols = 0;
  const void *dy = nullptr, *h = nullptr, *w = nullptr, *dh = nullptr;
  int64_t lddy = 0, ldh = 0, lddh = 0;
  const float* rstd = nullptr;
  void* dx = nullptr;
  int64_t lddx = 0;
  float* partial = nullptr;  // [grid][cols] sums of dW; nullptr: dW is not wanted
  float* dw = nullptr;
  int vec = 0;
};
constexpr int kNormGradMaxCols = 49152;  // the wide form keeps a row of dW sums in shared memory
cudaError_t prepare_fp8_norm();
// CTAs of the gradient kernel (its partial sums of dW take grid * cols floats).
int fp8_rmsnorm_backward_grid(int type, int64_t rows, int cols, int sm_count);
cudaError_t launch_fp8_rmsnorm_backward(int type, const NormGradParams& p, int grid, cudaStream_t stream);

}  // namespace sgemm_impl
