// Building blocks of the row and column operators (normalisation, activation
// gradients): 8-element vectors between memory and fp32 registers, block-wide
// reductions and 8-bit rounding.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "gemm_kernel.cuh"

namespace gb300 {

// Element types of the row operators' memory: DT_F32, DT_F16, DT_BF16 of the
// GEMM epilogue, and the two 8-bit types (outputs only).
enum : int { DT_E5M2 = 4 };

constexpr int kVec = 8;                // elements of one vector: 16 bytes of a 16-bit type

__host__ __device__ constexpr int elem_bytes(int dt) {
  return dt == DT_F32 ? 4 : (dt == DT_F16 || dt == DT_BF16) ? 2 : 1;
}

__device__ __forceinline__ void store_elem(void* p, long long i, int dt, float v) {
  if (dt == DT_F32) static_cast<float*>(p)[i] = v;
  else if (dt == DT_F16) static_cast<uint16_t*>(p)[i] = __half_as_ushort(__float2half_rn(v));
  else static_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// The raw bits of one vector of type DT, so that loads can be issued well
// before their values are converted.
template <int DT>
struct RawVec {
  uint4 q[DT == DT_F32 ? 2 : 1];
};

// Asynchronous copies of 16 bytes to shared memory, `bytes` of them read and the
// rest zero; a thread waits for its own, all but its latest n groups.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Wait until at most `n` of this thread's latest groups are in flight (n < 4).
__device__ __forceinline__ void copy_wait(int n) {
  if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// Elements [c, c + 8) of a row (p 16-byte aligned at c), those at or past `n`
// read as zero and not touched in memory.
template <int DT>
__device__ __forceinline__ RawVec<DT> load_raw(const void* row, int c, int n) {
  RawVec<DT> r;
  const uint8_t* const p = static_cast<const uint8_t*>(row) + (size_t)c * elem_bytes(DT);
  if (c + kVec <= n) {
    r.q[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (DT == DT_F32) r.q[1] = *reinterpret_cast<const uint4*>(p + 16);
  } else {
    uint32_t w[DT == DT_F32 ? 8 : 4];
#pragma unroll
    for (int i = 0; i < (DT == DT_F32 ? 8 : 4); ++i) w[i] = 0u;
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (c + i < n) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (c + i < n) w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    }
    r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (DT == DT_F32) r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void unpack(const RawVec<DT>& r, float (&v)[kVec]) {
  if constexpr (DT == DT_F32) {
    const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w,
                           r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = DT == DT_BF16 ? unpack_bf16x2(w[i]) : unpack_f16x2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ void load_vec(const void* row, int c, int n, float (&v)[kVec]) {
  unpack<DT>(load_raw<DT>(row, c, n), v);
}

// The same with the type known at run time (F32, F16 or BF16; uniform).
__device__ __forceinline__ void load_vec_dt(const void* row, int dt, int c, int n,
                                            float (&v)[kVec]) {
  if (dt == DT_F32) load_vec<DT_F32>(row, c, n, v);
  else if (dt == DT_F16) load_vec<DT_F16>(row, c, n, v);
  else load_vec<DT_BF16>(row, c, n, v);
}

// Two fp32 values -> two 8-bit codes in the low 16 bits (first in the low
// byte), rounded to nearest even, finite overflow clamped to the largest
// finite value, NaN kept.
__device__ __forceinline__ uint32_t pack_fp8x2(float lo, float hi, int dt) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE,
                                            dt == DT_E4M3 ? __NV_E4M3 : __NV_E5M2);
}

// Stores elements [c, c + 8) of a row (16-byte aligned at c for 16- and
// 32-bit types, 8-byte for 8-bit ones), none at or past `n`.  Uniform type.
__device__ __forceinline__ void store_vec(void* row, int dt, int c, int n,
                                          const float (&v)[kVec]) {
  uint8_t* const p = static_cast<uint8_t*>(row) + (size_t)c * elem_bytes(dt);
  if (dt == DT_F32) {
    if (c + kVec <= n) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (c + i < n) reinterpret_cast<float*>(p)[i] = v[i];
    }
  } else if (dt == DT_F16 || dt == DT_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = dt == DT_F16 ? pack_f16x2(v[2 * i], v[2 * i + 1]) : pack_bf16x2(v[2 * i], v[2 * i + 1]);
    if (c + kVec <= n) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (c + i < n) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  } else {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = pack_fp8x2(v[4 * i], v[4 * i + 1], dt) | pack_fp8x2(v[4 * i + 2], v[4 * i + 3], dt) << 16;
    if (c + kVec <= n) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (c + i < n) p[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
    }
  }
}

// ------------------------------------------------------------------ reductions

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over the block, the same value in every thread and in every run: lanes
// by a butterfly, warps in warp order.  `scratch` holds 32 floats; two calls
// in a row need different scratch (or a barrier between them).
__device__ __forceinline__ float block_sum(float v, float* scratch) {
  v = warp_sum(v);
  const int warps = (int)blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < warps; ++i) s += scratch[i];
  return s;
}

// Largest magnitude over the block, as the bits of a non-negative float: for
// those the order of the bits is the order of the values, and a NaN's are
// above infinity's, so a NaN anywhere in the row is what comes out.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* scratch) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  const int warps = (int)blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = 0;
  for (int i = 0; i < warps; ++i) m = max(m, scratch[i]);
  return m;
}

}  // namespace gb300
