// Host helpers of the row and column operators: argument checks and launches.
#pragma once

#include <cstdint>

#include "gemm_gb300.h"
#include "handle.h"
#include "rows.cuh"

namespace gb300host {

// Device type code of a C-ABI type.
inline int device_dt(int t) {
  switch (t) {
    case GEMM_F32: return gb300::DT_F32;
    case GEMM_F16: return gb300::DT_F16;
    case GEMM_BF16: return gb300::DT_BF16;
    case GEMM_E4M3: return gb300::DT_E4M3;
    default: return gb300::DT_E5M2;
  }
}

inline bool aligned_to(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

// One matrix argument: present where required, at least `cols` wide, its base
// and rows on 16-byte boundaries.
inline gemm_status_t check_matrix(const void* p, int64_t ld, int64_t cols, int dt) {
  if (!p || ld < cols) return GEMM_ERR_INVALID_ARG;
  if (!aligned16(p) || (ld * dtype_bytes(dt)) % 16 != 0) return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

#define GB300_CHECK(expr)                                     \
  do {                                                        \
    const gemm_status_t check_status = (expr);                \
    if (check_status != GEMM_OK) return check_status;         \
  } while (0)

// Raises `kern`'s dynamic shared-memory limit, once per handle (h->mu held).
inline gemm_status_t raise_smem(gemm_handle* h, const void* kern) {
  for (int i = 0; i < h->raised_count; ++i)
    if (h->raised[i] == kern) return GEMM_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           h->smem_optin - 1024) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (h->raised_count < gemm_handle::kMaxRaised) h->raised[h->raised_count++] = kern;
  return GEMM_OK;
}

// Launch on `stream`, allowed to be scheduled while the stream's previous
// kernel finishes (every kernel here waits for it before touching memory), in
// clusters of `cluster` blocks.
template <typename P>
gemm_status_t launch(void (*kern)(P), const P& params, int64_t grid, int threads, size_t smem,
                     struct CUstream_st* stream, int cluster = 1) {
  cudaLaunchConfig_t lc{};
  cudaLaunchAttribute attr[2];
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = reinterpret_cast<cudaStream_t>(stream);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  void* args[1] = {const_cast<P*>(&params)};
  if (cudaLaunchKernelExC(&lc, reinterpret_cast<const void*>(kern), args) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

}  // namespace gb300host
