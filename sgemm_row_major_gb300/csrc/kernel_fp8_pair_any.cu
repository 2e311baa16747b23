// kernel_fp8_pair_any.cu -- the CTA-pair 8-bit product, output form: rows of C or D at any alignment.
#include "kernel_fp8_pair.cuh"

namespace sgemm_impl {
SGEMM_DEFINE_FP8_PAIR(any, f8::kOutAny)
}  // namespace sgemm_impl
