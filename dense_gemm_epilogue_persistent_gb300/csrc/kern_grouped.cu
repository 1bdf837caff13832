// The kernel of products over groups of rows (grouped_kernel.cuh), compiled once per
// input width and form (rows, or the weights' gradients of 16-bit operands).
#include "grouped_kernel.cuh"
#include "kernels.h"

namespace gb300 {

template <int CG, int LEAN>
static const void* kernel() {
  return (const void*)&grouped_kernel<CG, GB300_AB, GB300_WEIGHTS != 0, LEAN>;
}

const void* GB300_GROUPED_NAME(GB300_AB, GB300_WEIGHTS)(int cta_group, int lean) {
#if GB300_AB == 2
  switch (lean) {
    case DT_F32: return cta_group == 1 ? kernel<1, DT_F32>() : kernel<2, DT_F32>();
    case DT_F16: return cta_group == 1 ? kernel<1, DT_F16>() : kernel<2, DT_F16>();
    case DT_BF16: return cta_group == 1 ? kernel<1, DT_BF16>() : kernel<2, DT_BF16>();
  }
#endif
  if (lean >= 0) return nullptr;
  return cta_group == 1 ? kernel<1, -1>() : kernel<2, -1>();
}

}  // namespace gb300
