// Host helpers of the row and column operators: argument checks and launches.
#pragma once

#include <cstdint>
#include <initializer_list>

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

// Whether an output, where there is one, lies where another of the call's tensors does.
inline bool same_place(const void* out, std::initializer_list<const void*> others) {
  for (const void* p : others)
    if (out && p == out) return true;
  return false;
}

#define GB300_CHECK(expr)                                     \
  do {                                                        \
    const gemm_status_t check_status = (expr);                \
    if (check_status != GEMM_OK) return check_status;         \
  } while (0)

inline bool is_activation(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }

// Sizes the kernels index with 32 bits: what they add to an index on the way to its
// bound (the rest of the last tile, whose width need not divide 2^31; a vector's
// end; a cluster's shares of the rows) stays below 2^31.
inline bool is_extent(int64_t v) { return v >= 0 && v <= INT32_MAX - 8192; }
// Tensor-map strides below 2^40 bytes.
inline bool map_ok(int64_t ld, int64_t rows, int dt) {
  return (double)ld * dtype_bytes(dt) * (double)rows < 1099511627776.0;
}

// One A or B operand: `inner` contiguous elements a row, `rows` rows.
inline gemm_status_t check_operand(const void* p, int64_t ld, int64_t inner, int64_t rows, int dt) {
  GB300_CHECK(check_matrix(p, ld, inner, dt));
  return map_ok(ld, rows, dt) ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

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

// linear.cu: dz = dd act'(z) over the rows of groups, and each group's bias gradient
// (either output may be null); the arguments have been checked.
struct GroupedActGrad {
  int64_t M, N, groups;
  gemm_dtype_t type, dbias_type;
  gemm_activation_t activation;
  const int32_t* offsets;
  const void* dd; int64_t lddd;
  const void* z; int64_t ldz;
  void* dz; int64_t lddz;
  void* dbias;
};
gemm_status_t grouped_act_grad(gemm_handle* h, const GroupedActGrad& g, struct CUstream_st* stream);

}  // namespace gb300host
