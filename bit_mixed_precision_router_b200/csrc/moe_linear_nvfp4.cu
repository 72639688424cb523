// moe_linear_w4 for NVFP4 matrices (the kernel: moe_linear.cuh).
#include "moe_linear.cuh"

namespace moe {

cudaError_t linear_nvfp4(const LinearArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? pick_linear<true, MOE_FMT_NVFP4>(a, st) : pick_linear<false, MOE_FMT_NVFP4>(a, st);
}

}  // namespace moe
