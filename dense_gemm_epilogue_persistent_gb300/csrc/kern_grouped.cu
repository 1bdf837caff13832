// The kernel of products over groups of rows (grouped_kernel.cuh), compiled once per
// input width and form (of the rows; of 16-bit operands also the weights' gradients, and both
// gradients in one launch).
#include "grouped_kernel.cuh"
#include "kernels.h"

namespace gb300 {

template <int CG, int LEAN>
static const void* kernel() {
  return (const void*)&grouped_kernel<CG, GB300_AB, GB300_FORM, LEAN>;
}

const void* GB300_GROUPED_NAME(GB300_AB, GB300_FORM)(int cta_group, int lean) {
#if GB300_AB == 2
  switch (lean) {
    case DT_F32: return cta_group == 1 ? kernel<1, DT_F32>() : kernel<2, DT_F32>();
    case DT_F16: return cta_group == 1 ? kernel<1, DT_F16>() : kernel<2, DT_F16>();
    case DT_BF16: return cta_group == 1 ? kernel<1, DT_BF16>() : kernel<2, DT_BF16>();
  }
#endif
#if GB300_FORM != 2
  if (lean < 0) return cta_group == 1 ? kernel<1, -1>() : kernel<2, -1>();
#endif
  return nullptr;
}

}  // namespace gb300
