// The kernel of products over groups of rows (grouped_kernel.cuh), compiled once per
// input width.
#include "grouped_kernel.cuh"
#include "kernels.h"

namespace gb300 {

const void* GB300_GROUPED_NAME(GB300_AB)(int cta_group, int form) {
#if GB300_AB == 2
  if (form == kGroupedWeights)
    return cta_group == 1 ? (const void*)&grouped_kernel<1, 2, kGroupedWeights>
                          : (const void*)&grouped_kernel<2, 2, kGroupedWeights>;
  if (form == kGroupedPlainRows)
    return cta_group == 1 ? (const void*)&grouped_kernel<1, 2, kGroupedPlainRows>
                          : (const void*)&grouped_kernel<2, 2, kGroupedPlainRows>;
#endif
  if (form != kGroupedRows) return nullptr;
  return cta_group == 1 ? (const void*)&grouped_kernel<1, GB300_AB, kGroupedRows>
                        : (const void*)&grouped_kernel<2, GB300_AB, kGroupedRows>;
}

}  // namespace gb300
