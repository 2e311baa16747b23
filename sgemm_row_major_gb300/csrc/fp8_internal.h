// fp8_internal.h -- host-side declarations of the 8-bit operators (sgemm_fp8.h).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "sgemm_fp8.h"

namespace sgemm_impl {

// What an entry point needs of the current device (set up by the first call on it, the 8-bit kernels
// by the first that needs them; api.cu).
struct CallDevice {
  int sm_count = 0;
  int pair_clusters = 0;
  unsigned* fault = nullptr;
  unsigned long long* bounds = nullptr;
  cudaMemPool_t pool = nullptr;
};
int call_device(CallDevice* out);  // an sgemm_status

// Where the debug build records an index that falls outside its buffer (in_range, device_utils.cuh).
struct Guard {
  unsigned* fault = nullptr;
  unsigned long long* word = nullptr;
};

// ---- quantiser (kernel_fp8_quant.cu)
struct QuantParams {
  const void* x = nullptr;
  int64_t rows = 0, cols = 0, ldx = 0;
  uint8_t* q = nullptr;
  int64_t ldq = 0;
  float* s = nullptr;
  int64_t lds = 0;
  int format = 0;
  int x_vec = 0;  // 1: rows of X start at multiples of 16 bytes
  Guard guard;
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
  int vec = 0;  // 1: rows of all matrices start at multiples of 16 bytes and hold whole chunks of 8
  Guard guard;
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
  uint64_t timeout_ns = 0;
  unsigned* fault = nullptr;
  Guard guard;
};
constexpr int kNormGradMaxCols = 49152;  // the wide form keeps a row of dW sums in shared memory
cudaError_t prepare_fp8_norm();
// CTAs of the gradient kernel (its partial sums of dW take grid * cols floats).
int fp8_rmsnorm_backward_grid(int type, int64_t rows, int cols, bool vec, int sm_count);
cudaError_t launch_fp8_rmsnorm_backward(int type, const NormGradParams& p, int grid, cudaStream_t stream);

// ---- product (kernel_fp8_pair.cuh, kernel_fp8_short.cu)

// Scales of one operand of a product: of row (or column) i of op(X) in group g of 128 k,
// p[(i >> shift) * si + g * sk].
struct Fp8Scales {
  const float* p = nullptr;
  int64_t si = 0, sk = 0;
  int shift = 0;  // 0: one per row (column), 7: one per 128
};

// D = alpha * op(A) op(B) + beta * C
struct Fp8Out {
  int M = 0, N = 0;
  float alpha = 1.0f, beta = 0.0f;
  const void* C = nullptr;
  void* D = nullptr;
  int64_t ldc = 0, ldd = 0;
  int bf16 = 0;  // type of C and D
  int vec = 0;   // 1: rows of C and D start at multiples of 16 bytes
  Guard guard;
};

struct Fp8PairParams {
  Fp8Out out;
  int K = 0;
  Fp8Scales sa, sb;
  int a_mn = 0, b_mn = 0;  // 1: the stored rows run along M (N), not along K
  uint32_t idesc = 0;
  int tiles_m = 0, tiles_n = 0, clusters = 0;
  uint64_t timeout_ns = 0;
  unsigned* fault = nullptr;
};
constexpr int kFp8PairStages = 5, kFp8PairThreads = 384;
int64_t fp8_pair_smem(bool cols);  // dynamic shared memory; cols: B has a scale per column
constexpr int kFp8PairTiles[] = {256, 128, 64};  // the tile widths there are kernels for
// One translation unit per form of the output: beta == 0 and aligned rows of whole 16 bytes, beta != 0 and
// aligned rows, anything.
#define SGEMM_DECLARE_FP8_PAIR(name)                                                               \
  cudaError_t prepare_fp8_pair_##name();                                                           \
  cudaError_t launch_fp8_pair_##name(int tile_n, const CUtensorMap& mapA, const CUtensorMap& mapB, \
                                     const CUtensorMap& mapD, const Fp8PairParams& p, cudaStream_t stream);
SGEMM_DECLARE_FP8_PAIR(plain)
SGEMM_DECLARE_FP8_PAIR(add)
SGEMM_DECLARE_FP8_PAIR(any)
#undef SGEMM_DECLARE_FP8_PAIR

// The longer of M and N runs along the tensor-core rows (`l`), the other along the columns (`s`).
struct Fp8ShortParams {
  Fp8Out out;
  int K = 0, L = 0, S = 0;
  int trans = 0;  // 1: l runs along N (D_sl), 0: along M (D_ls)
  Fp8Scales sl, ss;
  int l_mn = 0, s_mn = 0;
  uint32_t idesc = 0;
  int tile_s = 0, tiles_l = 0, tiles_s = 0, split = 1, stages = 0, stage_bytes = 0;
  uint64_t timeout_ns = 0;
  unsigned* fault = nullptr;
};
cudaError_t prepare_fp8_short();
constexpr int kFp8ShortTiles[] = {16, 32, 64, 128};  // the tile widths there are kernels for
constexpr int kFp8ShortMaxStages = 12, kFp8ShortThreads = 256;
size_t fp8_short_smem(int tile_s, int stages, int stage_bytes);
cudaError_t launch_fp8_short(const CUtensorMap& mapL, const CUtensorMap& mapS, const Fp8ShortParams& p,
                             cudaStream_t stream);

// ---- mixture of experts for a few tokens (kernel_fp8_moe.cu)
constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 1024, kMoeMaxTopK = 16;
struct MoeParams {
  int tokens = 0, hidden = 0, inner = 0, experts = 0, top_k = 0, renormalize = 0;
  const float* logits = nullptr;
  int64_t ldl = 0;
  const float* sx = nullptr;              // scales of X, row stride ldsx
  int64_t ldsx = 0;
  const float *sg = nullptr, *su = nullptr, *sd = nullptr;  // scales of gate, up, down
  int64_t ldsg = 0, ldsu = 0, ldsd = 0, stride_sg = 0, stride_su = 0, stride_sd = 0;
  uint8_t* h = nullptr;                   // inner values: slot j has rows 2j (hi) and 2j + 1 (lo * 16) of `inner` codes
  float* sh = nullptr;                    // [slots][h_groups], one scale per 64 of them
  int h_groups = 0;
  void* y = nullptr;
  int64_t ldy = 0;
  int bf16 = 0;
  int up_stages = 0, down_stages = 0, down_grid = 0;
  int* arrived = nullptr;                 // [ceil(hidden / 128)] CTAs whose sums are in `part`
  float* part = nullptr;                  // [2 * down_grid][tokens][128]
  int many = 0;                           // 1: many units per CTA: the kernels run one after the other
  int* route = nullptr;                   // the routing, left by the first kernel where `many`
  int active_max = 0, slots_max = 0;      // bounds of the routing arrays
  Guard guard;
  uint64_t timeout_ns = 0;
  unsigned* fault = nullptr;
};
struct MoeMaps {
  CUtensorMap x, gate, up, h, down;
};
cudaError_t prepare_fp8_moe();
// Fills the launch shape (stages, grid) of p.
void shape_fp8_moe(MoeParams* p, int sm_count);
cudaError_t launch_fp8_moe(const MoeMaps& maps, const MoeParams& p, int sm_count, cudaStream_t stream);

// Map over `outer` rows of `inner` 8-bit codes (row stride ld bytes, a multiple of 16): boxes of 128
// codes x box_outer rows, 128-byte swizzle, zeros outside.
cudaError_t encode_fp8_map(const void* base, int64_t inner, int64_t outer, int64_t ld, int box_outer,
                           CUtensorMap* map);
// Map over D (`rows` x `cols` FP32 or BF16, row stride ld elements, 16-byte aligned rows of whole 16 bytes, as
// TMA writes the rest of a unit too): boxes of 32 x 32, swizzled by their rows' width.
cudaError_t encode_out_map(const void* base, int64_t cols, int64_t rows, int64_t ld, bool bf16, CUtensorMap* map);
// The same as encode_fp8_map over `products` such matrices `stride` bytes apart (a multiple of 16).
cudaError_t encode_fp8_maps(const void* base, int64_t inner, int64_t outer, int64_t ld, int64_t products,
                            int64_t stride, int box_outer, CUtensorMap* map);
// Rows of `cols` codes copied to rows `ldd` apart (any alignment of the source).
cudaError_t launch_fp8_repack(const void* src, int64_t ld, int64_t rows, int64_t cols, void* dst, int64_t ldd,
                              const Guard& guard, cudaStream_t stream);
// D = beta * C (alpha == 0 or K == 0).
cudaError_t launch_fp8_scale(const Fp8Out& o, cudaStream_t stream);

}  // namespace sgemm_impl
