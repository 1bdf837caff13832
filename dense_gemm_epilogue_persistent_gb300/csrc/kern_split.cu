// The split-K kernel of the linear layer (split_kernel.cuh), one unit for the
// three input widths.
#include "kernels.h"
#include "split_kernel.cuh"

namespace gb300 {

const void* split_kernel_for(int ab_bytes) {
  switch (ab_bytes) {
    case 2: return (const void*)&linear_split_kernel<2>;
    case 1: return (const void*)&linear_split_kernel<1>;
    case 4: return (const void*)&linear_split_kernel<4>;
  }
  return nullptr;
}

}  // namespace gb300
