// api_fp8.cu -- the C ABI of the 8-bit operators (sgemm_fp8.h): argument checks, workspace and launches.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "fp8_internal.h"
#include "sgemm_fp8.h"
#include "sgemm_internal.h"

using namespace sgemm_impl;

namespace {

constexpr int64_t kMaxDim = INT_MAX - 1024;  // column indices of the kernels' last chunks stay below 2^31

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int type_size(int type) { return type == SGEMM_BF16 ? 2 : 4; }
bool known_type(int type) { return type == SGEMM_F32 || type == SGEMM_BF16; }
bool known_format(int f) { return f == SGEMM_FP8_E4M3 || f == SGEMM_FP8_E5M2; }

// Rows of 16-byte vectors: the base and the row stride in bytes are multiples of 16 (a NULL matrix is not read).
bool rows16(const void* p, int64_t ld, int size) { return !p || (aligned(p, 16) && ld * size % 16 == 0); }

int launch_status(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : record_cuda_failure(e); }

}  // namespace

extern "C" {

int sgemm_fp8_quantize(int64_t rows, int64_t cols, const void* X, int type, int64_t ldx, int format, int block_rows,
                       int block_cols, void* codes, int64_t ldq, float* scale, int64_t lds,
                       struct CUstream_st* stream) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  const bool work = rows > 0 && cols > 0;
  if (!known_type(type)) return -4;
  if (work && (!X || !aligned(X, type_size(type)))) return -3;
  if (ldx < std::max<int64_t>(1, cols)) return -5;
  if (!known_format(format)) return -6;
  if (block_rows != 1 && block_rows != 128) return -7;
  if ((block_cols != 1 && block_cols != 128) || (block_rows == 1 && block_cols == 1)) return -8;
  if (work && !codes) return -9;
  if (ldq < std::max<int64_t>(1, cols)) return -10;
  if (work && (!scale || !aligned(scale, 4))) return -11;
  if (lds < std::max<int64_t>(1, ceil_div(cols, block_cols))) return -12;
  if (!work) return SGEMM_OK;
  if (rows > kMaxDim || cols > kMaxDim || ceil_div(rows, 128) * ceil_div(cols, 128) > INT_MAX)
    return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  const int s = call_device(&dev);
  if (s != SGEMM_OK) return s;
  QuantParams p;
  p.x = X;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.q = static_cast<uint8_t*>(codes);
  p.ldq = ldq;
  p.s = scale;
  p.lds = lds;
  p.format = format;
  p.vec = rows16(X, ldx, type_size(type)) && aligned(codes, 8) && ldq % 8 == 0;
  return launch_status(launch_fp8_quantize(type, block_rows, block_cols, p, reinterpret_cast<cudaStream_t>(stream)));
}

int sgemm_fp8_rmsnorm(int64_t rows, int64_t cols, int type, const void* X, int64_t ldx, const void* R, int64_t ldr,
                      const void* W, float eps, void* H, int64_t ldh, void* Y, int64_t ldy, void* codes, int64_t ldq,
                      float* scale, int64_t lds, float* rstd, struct CUstream_st* stream) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  if (!known_type(type)) return -3;
  const int size = type_size(type);
  const bool work = rows > 0 && cols > 0;
  const int64_t min_ld = std::max<int64_t>(1, cols);
  if (work && (!X || !aligned(X, size))) return -4;
  if (ldx < min_ld) return -5;
  if (R && !aligned(R, size)) return -6;
  if (R && ldr < min_ld) return -7;
  if (work && (!W || !aligned(W, size))) return -8;
  if (!(eps >= 0.0f)) return -9;
  if (H && !aligned(H, size)) return -10;
  if (H && ldh < min_ld) return -11;
  if (Y && !aligned(Y, size)) return -12;
  if (Y && ldy < min_ld) return -13;
  if (codes && ldq < min_ld) return -15;
  if (work && codes && (!scale || !aligned(scale, 4))) return -16;
  if (codes && lds < std::max<int64_t>(1, ceil_div(cols, 128))) return -17;
  if (rstd && !aligned(rstd, 4)) return -18;
  if (!work) return SGEMM_OK;
  if (rows > kMaxDim || cols > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  const int s = call_device(&dev);
  if (s != SGEMM_OK) return s;
  NormParams p;
  p.rows = rows;
  p.cols = (int)cols;
  p.x = X;
  p.ldx = ldx;
  p.r = R;
  p.ldr = ldr;
  p.w = W;
  p.eps = eps;
  p.h = H;
  p.ldh = ldh;
  p.y = Y;
  p.ldy = ldy;
  p.q = static_cast<uint8_t*>(codes);
  p.ldq = ldq;
  p.s = scale;
  p.lds = lds;
  p.rstd = rstd;
  p.vec = rows16(X, ldx, size) && rows16(R, ldr, size) && rows16(W, 0, size) && rows16(H, ldh, size) &&
          rows16(Y, ldy, size) && (!codes || (aligned(codes, 8) && ldq % 8 == 0));
  return launch_status(launch_fp8_rmsnorm(type, p, reinterpret_cast<cudaStream_t>(stream)));
}

int sgemm_fp8_rmsnorm_backward(int64_t rows, int64_t cols, int type, const void* dY, int64_t lddy, const void* H,
                               int64_t ldh, const void* W, const float* rstd, const void* dH, int64_t lddh, void* dX,
                               int64_t lddx, float* dW, struct CUstream_st* stream_) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  if (!known_type(type)) return -3;
  const int size = type_size(type);
  const bool work = rows > 0 && cols > 0;
  const int64_t min_ld = std::max<int64_t>(1, cols);
  if (work && (!dY || !aligned(dY, size))) return -4;
  if (lddy < min_ld) return -5;
  if (work && (!H || !aligned(H, size))) return -6;
  if (ldh < min_ld) return -7;
  if (work && (!W || !aligned(W, size))) return -8;
  if (work && (!rstd || !aligned(rstd, 4))) return -9;
  if (dH && !aligned(dH, size)) return -10;
  if (dH && lddh < min_ld) return -11;
  if (work && (!dX || !aligned(dX, size))) return -12;
  if (lddx < min_ld) return -13;
  if (dW && !aligned(dW, 4)) return -14;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (cols == 0 || (rows == 0 && !dW)) return SGEMM_OK;
  if (rows > kMaxDim || cols > kNormGradMaxCols) return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  const int s = call_device(&dev);
  if (s != SGEMM_OK) return s;
  if (rows == 0) return launch_status(cudaMemsetAsync(dW, 0, (size_t)cols * 4, stream));  // a sum of nothing
  NormGradParams p;
  p.rows = rows;
  p.cols = (int)cols;
  p.dy = dY;
  p.lddy = lddy;
  p.h = H;
  p.ldh = ldh;
  p.w = W;
  p.rstd = rstd;
  p.dh = dH;
  p.lddh = lddh;
  p.dx = dX;
  p.lddx = lddx;
  p.dw = dW;
  p.vec = rows16(dY, lddy, size) && rows16(H, ldh, size) && rows16(W, 0, size) && rows16(dH, lddh, size) &&
          rows16(dX, lddx, size);
  const int grid = fp8_rmsnorm_backward_grid(type, rows, (int)cols, dev.sm_count);
  if (dW) {
    void* ws = nullptr;
    cudaError_t e = cudaMallocFromPoolAsync(&ws, (size_t)grid * cols * 4, dev.pool, stream);
    if (e != cudaSuccess) {
      record_cuda_failure(e);
      return e == cudaErrorMemoryAllocation ? SGEMM_ERR_NOMEM : SGEMM_ERR_CUDA;
    }
    p.partial = static_cast<float*>(ws);
  }
  cudaError_t e = launch_fp8_rmsnorm_backward(type, p, grid, stream);
  if (p.partial) {
    const cudaError_t ef = cudaFreeAsync(p.partial, stream);
    if (e == cudaSuccess) e = ef;
  }
  return launch_status(e);
}

}  // extern "C"
