// Persistent-GEMM variants with the linear layer's epilogue (scales, bias,
// activation, residual; gemm_kernel.cuh, EPI = 1) and, at 16 bits, for two
// products in one launch (EPI = 2): clusters of one CTA group.  Compiled once
// per input width, GB300_AB = 2 (fp16/bf16), 1 (fp8) or 4 (tf32), per count of
// epilogue warps per tensor-memory lane quarter, GB300_EPW = 1 or 2, and per
// GB300_EPI = 1 or 2.
#include "gemm_kernel.cuh"
#include "kernels.h"

namespace gb300 {

const void* GB300_LINEAR_NAME(GB300_AB, GB300_EPW, GB300_EPI)(int cta_group, int ka) {
  if (cta_group == 1 && ka == 1)
    return (const void*)&persistent_gemm_kernel<1, GB300_AB, 1, 1, 1, GB300_EPW, 0, GB300_EPI>;
  if (cta_group == 1 && ka == 2)
    return (const void*)&persistent_gemm_kernel<1, GB300_AB, 2, 1, 1, GB300_EPW, 0, GB300_EPI>;
  if (cta_group == 2 && ka == 2)
    return (const void*)&persistent_gemm_kernel<2, GB300_AB, 2, 1, 1, GB300_EPW, 0, GB300_EPI>;
  return nullptr;
}

}  // namespace gb300
