// kernel_fp8_pair_add.cu -- the CTA-pair 8-bit product, output form: beta != 0, aligned rows.
#include "kernel_fp8_pair.cuh"

namespace sgemm_impl {
SGEMM_DEFINE_FP8_PAIR(add, f8::kOutAdd)
}  // namespace sgemm_impl
