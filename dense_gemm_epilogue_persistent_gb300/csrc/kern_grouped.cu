// The kernel of products over groups of rows (grouped_kernel.cuh), compiled once per
// input width.
#include "grouped_kernel.cuh"
#include "kernels.h"

namespace gb300 {

const void* GB300_GROUPED_NAME(GB300_AB)(int cta_group, bool weights) {
#if GB300_AB == 2
  if (weights)
    return cta_group == 1 ? (const void*)&grouped_kernel<1, 2, true>
                          : (const void*)&grouped_kernel<2, 2, true>;
#endif
  if (weights) return nullptr;
  return cta_group == 1 ? (const void*)&grouped_kernel<1, GB300_AB, false>
                        : (const void*)&grouped_kernel<2, GB300_AB, false>;
}

}  // namespace gb300
