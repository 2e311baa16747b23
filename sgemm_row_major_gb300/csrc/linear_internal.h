// linear_internal.h -- host-side declarations of the operators on BF16 layers (sgemm_linear.h).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8_internal.h"
#include "sgemm_linear.h"

namespace sgemm_impl {

// What an entry point of this part needs of the current device (its kernels are set up by the first call; api.cu).
int linear_device(CallDevice* out);  // an sgemm_status

// What happens to a product's sums: bias, activation, residual, the output and what is kept of the sums.
struct LinearKept {
  void* data = nullptr;
  float* scale = nullptr;
  int64_t ld = 0, lds = 0;
  int vec = 0;                   // 1: rows start at multiples of 16 bytes
};
struct LinearOut {
  const void* bias = nullptr;    // N values or nullptr
  const void* residual = nullptr;
  int64_t ldr = 0;
  int act = 0;
  int keep = 0;                  // 0: nothing, 1: BF16, 2: 8-bit
  LinearKept kept[2];            // of A and B
  int bias_vec = 0, r_vec = 0;   // 1: 16-byte aligned (rows)
  int kept_vec8[2] = {0, 0};     // 1: rows of a BF16 kept matrix start at multiples of 8 bytes
  Guard guard;
};

// One product of a launch: D = A0 B0 (+ A1 B1 with two segments of K); gated: B0 and B1 are gate and up, D is H.
struct LinearJob {
  int M = 0, N = 0;              // rows and columns of D
  void* d = nullptr;
  int64_t ldd = 0;
  int d_tma = 0;                 // 1: rows start at multiples of 16 bytes: TMA writes the whole 16 bytes of them
  int d_vec = 0;                 // 1: rows start at multiples of 8 bytes (BF16) or 16 bytes (FP32)
  int f32 = 0;
  int tiles_m = 0, tiles_n = 0;
  int k_tiles = 0, segments = 1; // of 64 k, per segment
  int fold0 = 0, fold = 1;       // K tiles that are summed in the first accumulator, and in each further one
  int a_mn = 0, b_mn = 0;        // 1: the stored rows run along M (N), not along K
  uint32_t idesc = 0;
  int a[2] = {0, 0}, b[2] = {0, 0};  // maps of the operands
  // split > 1 (pair kernel): the K tiles of a tile are shared by that many units, each of which writes its sums to an FP32
  // matrix of its own, `rows_apart` rows below the one before (D then stands for all of them: M = split * rows_apart)
  int split = 1, rows_apart = 0;
};
constexpr int kLinearJobs = 3;
struct LinearMaps {
  CUtensorMap op[6], d[kLinearJobs], kept[2];
};

struct LinearPairParams {
  LinearOut out;
  LinearJob job[kLinearJobs];    // their tiles one behind the other
  int jobs = 1, clusters = 0;
  uint64_t timeout_ns = 0;
  unsigned* fault = nullptr;
};
constexpr int kLinearPairThreads = 384;
constexpr int kLinearPairTiles[] = {256, 128, 64};
// Columns of the pieces of D that TMA writes (BF16; FP32: 32), which the epilogue takes at a time.  With the 128 sums of a
// 256-wide tile in registers 64 columns at a time spill.
constexpr int linear_pair_box(int tile_n, bool gated, bool fold) {
  return tile_n / (gated ? 4 : 2) >= 64 && !(fold && !gated && tile_n == 256) ? 64 : 32;
}
int linear_pair_stages(int tile_n);
int64_t linear_pair_smem(int tile_n);
cudaError_t prepare_linear_pair();
// kFold: some job has an FP32 output, keeps 8-bit values or has a long sum.  kShared: some job's K is shared; nothing follows the products.
enum class LinearPairForm { kWhole, kFold, kShared };
cudaError_t launch_linear_pair(int tile_n, bool gated, LinearPairForm form, const LinearMaps& maps, const LinearPairParams& p, cudaStream_t stream);

// The columns of D run along the tensor core's rows (B's tile of 128), its rows along the columns.
struct LinearShortParams {
  LinearOut out;
  LinearJob job;
  int tile_s = 0, split = 1, stages = 0, stage_bytes = 0;
  uint64_t timeout_ns = 0;
  unsigned* fault = nullptr;
};
constexpr int kLinearShortTiles[] = {16, 32, 64, 128};
constexpr int kLinearShortMaxStages = 12, kLinearShortThreads = 256;
int64_t linear_short_smem(int tile_s, bool gated, int stages, int stage_bytes);
cudaError_t prepare_linear_short();
cudaError_t launch_linear_short(bool gated, const LinearMaps& maps, const LinearShortParams& p, cudaStream_t stream);

// The sums of products whose K was shared: each job's `split` matrices added in order, then the epilogue (of the first job).
constexpr int kLinearMostShares = 32;  // units of a tile
struct LinearJoin {
  const float* sums = nullptr;
  int64_t ld = 0;                // row stride of the sums
  int split = 1, rows_apart = 0;
  LinearJob job;                 // M, N and D of the product
  int64_t blocks = 0;            // of the launch
  int parts = 1;                 // threads that share the sums of an element
};
struct LinearJoinParams {
  LinearJoin part[kLinearJobs];
  LinearOut out;
};
cudaError_t launch_linear_join(LinearJoinParams& p, cudaStream_t stream);

// The elementwise part of the backward passes (kernel_linear_grad.cu).
struct LinearKeptIn {
  const void* data = nullptr;    // nullptr: not read
  const float* scale = nullptr;  // nullptr: BF16
  int64_t ld = 0, lds = 0;
  int vec = 0;                   // 1: chunks of 8 elements can be read at once (not looked at by the copies)
};
struct LinearGradParams {
  int64_t rows = 0;
  int cols = 0;
  const void* dy = nullptr;
  int64_t lddy = 0;
  LinearKeptIn a, b;             // b: gated
  int act = 0;
  void *da = nullptr, *db = nullptr, *h = nullptr;  // nullptr: not wanted (da and db: aligned rows)
  int64_t ldd = 0, ldh = 0;
  float* dbias = nullptr;        // nullptr: not wanted
  int strip = 0, row_blocks = 0; // columns of a CTA; CTAs that share the rows
  int joined = 0;                // dbias: 1: a cluster's CTAs add their sums, 0: a second kernel those in `partial`
  float* partial = nullptr;      // [row_blocks][cols]
  int vec = 0;                   // 1: chunks of 8 columns can be read and written at once
  Guard guard;
};
void shape_linear_grad(LinearGradParams* p, bool clusters, int sm_count);  // fills strip, row_blocks and joined
cudaError_t launch_linear_grad(const LinearGradParams& p, cudaStream_t stream);

// Stored matrices as aligned BF16 rows (ldd a multiple of 8): BF16 of any alignment copied, 8-bit values times their scales.
struct LinearExpand {
  LinearKeptIn m;
  int64_t rows = 0;
  int cols = 0;
  void* dst = nullptr;
  int64_t ldd = 0;
  int64_t blocks = 0;            // of the launch
};
struct LinearExpandParams {
  LinearExpand part[3];
  Guard guard;
};
cudaError_t launch_linear_expand(LinearExpandParams& p, cudaStream_t stream);

// Map over `outer` rows of `inner` BF16 values (row stride ld elements, a multiple of 8): boxes of 64 x box_outer,
// 128-byte swizzle, zeros outside.
cudaError_t encode_linear_map(const void* base, int64_t inner, int64_t outer, int64_t ld, int box_outer, CUtensorMap* map);

// Map over D (`rows` x `cols` BF16 or FP32, row stride ld elements, rows that start at multiples of 16 bytes; what a row holds
// beyond whole 16 bytes is left out, as TMA would write behind it): boxes of box_cols x 32, rows of 64 or 128 bytes with the swizzle of that width.
cudaError_t encode_linear_out_map(const void* base, int64_t cols, int64_t rows, int64_t ld, bool bf16, int box_cols, CUtensorMap* map);

}  // namespace sgemm_impl
