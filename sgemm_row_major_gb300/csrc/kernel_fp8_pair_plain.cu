// kernel_fp8_pair_plain.cu -- the CTA-pair 8-bit product, output form: beta == 0, aligned rows of whole 16 bytes.
#include "kernel_fp8_pair.cuh"

namespace sgemm_impl {
SGEMM_DEFINE_FP8_PAIR(plain, f8::kOutPlain)

int64_t fp8_pair_smem(bool cols) { return cols ? f8::ScaleCfg<true>::kSmem : f8::ScaleCfg<false>::kSmem; }
}  // namespace sgemm_impl
