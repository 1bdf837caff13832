// Root-mean-square normalisation fused with the residual's addition and an
// 8-bit output, and its backward pass (include/gemm_gb300.h).
#include <algorithm>
#include <cstdint>

#include "gemm_gb300.h"
#include "handle.h"
#include "rows.cuh"
#include "rows_host.h"

namespace gb300 {

struct NormParams {
  long long ldx, ldr, ldh, ldy;     // row strides in elements
  const void* x;
  const void* r;                    // residual or null
  void* h;                          // x + residual, or null
  const void* w;
  void* y;
  float* scale;                     // per-row scale of an 8-bit y
  float* rstd;                      // or null
  int M, H;
  int w_dt, y_dt;
  float eps, inv_h;
};

// The smallest largest-magnitude a row's scale is derived from: below it the
// scale and its reciprocal would leave fp32's normal range.
constexpr float kAmaxFloor = 7.888609052210118e-31f;    // 2^-100

__device__ __forceinline__ float largest_fp8(int dt) { return dt == DT_E4M3 ? 448.f : 57344.f; }

// A row of any length: one block, three passes over the row (sum of squares,
// largest output magnitude where the output is 8-bit, outputs).  The later
// passes read the row again (from L2: a row is far smaller).  H and y are
// written in the last pass only, each element by the thread that has just
// read that element of x and the residual, so either may be updated in place.
template <int DT>
__global__ void __launch_bounds__(1024)
rmsnorm_any_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[32];
  __shared__ uint32_t maxs[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const long long row = blockIdx.x;
  constexpr int es = elem_bytes(DT);
  const uint8_t* const x = static_cast<const uint8_t*>(p.x) + row * p.ldx * es;
  const uint8_t* const r =
      p.r ? static_cast<const uint8_t*>(p.r) + row * p.ldr * es : nullptr;
  const int step = (int)blockDim.x * kVec;
  auto read = [&](int c, float (&v)[kVec]) {
    load_vec<DT>(x, c, p.H, v);
    if (r) {
      float u[kVec];
      load_vec<DT>(r, c, p.H, u);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] += u[i];
    }
  };

  float ss = 0.f;
  for (int c = threadIdx.x * kVec; c < p.H; c += step) {
    float v[kVec];
    read(c, v);
#pragma unroll
    for (int i = 0; i < kVec; ++i) ss = fmaf(v[i], v[i], ss);
  }
  const float rstd = 1.f / sqrtf(block_sum(ss, sums) * p.inv_h + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  auto normed = [&](int c, float (&v)[kVec]) {
    float w[kVec];
    load_vec_dt(p.w, p.w_dt, c, p.H, w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = v[i] * rstd * w[i];
  };

  float inv = 1.f;
  const bool fp8 = p.y_dt >= DT_E4M3;
  if (fp8) {
    uint32_t big = 0;
    for (int c = threadIdx.x * kVec; c < p.H; c += step) {
      float v[kVec];
      read(c, v);
      normed(c, v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) big = max(big, abs_bits(v[i]));
    }
    big = max(block_max(big, maxs), __float_as_uint(kAmaxFloor));
    const float amax = __uint_as_float(big), top = largest_fp8(p.y_dt);
    inv = top / amax;
    if (threadIdx.x == 0) p.scale[row] = amax / top;
  }
  uint8_t* const y = static_cast<uint8_t*>(p.y) + row * p.ldy * elem_bytes(p.y_dt);
  uint8_t* const h = p.h ? static_cast<uint8_t*>(p.h) + row * p.ldh * es : nullptr;
  for (int c = threadIdx.x * kVec; c < p.H; c += step) {
    float v[kVec];
    read(c, v);
    if (h) store_vec(h, DT, c, p.H, v);
    normed(c, v);
    if (fp8) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] *= inv;
    }
    store_vec(y, p.y_dt, c, p.H, v);
  }
}

// ------------------------------------------------------------------ backward

struct NormBwdParams {
  long long lddy, ldh, lddh, lddx;
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dh;                   // gradient reaching h directly, or null
  void* dx;
  void* dw;
  int M, H;
  int w_dt, dw_dt;
  float inv_h;
};

// dx of a row of any length: one block, two passes (mean of dy w n, outputs);
// dx may be dh.
template <int DT>
__global__ void __launch_bounds__(1024)
rmsnorm_bwd_any_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float sums[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const long long row = blockIdx.x;
  constexpr int es = elem_bytes(DT);
  const uint8_t* const dy = static_cast<const uint8_t*>(p.dy) + row * p.lddy * es;
  const uint8_t* const h = static_cast<const uint8_t*>(p.h) + row * p.ldh * es;
  const uint8_t* const dh =
      p.dh ? static_cast<const uint8_t*>(p.dh) + row * p.lddh * es : nullptr;
  uint8_t* const dx = static_cast<uint8_t*>(p.dx) + row * p.lddx * es;
  const float rstd = p.rstd[row];
  const int step = (int)blockDim.x * kVec;
  float dot = 0.f;
  for (int c = threadIdx.x * kVec; c < p.H; c += step) {
    float g[kVec], n[kVec], w[kVec];
    load_vec<DT>(dy, c, p.H, g);
    load_vec<DT>(h, c, p.H, n);
    load_vec_dt(p.w, p.w_dt, c, p.H, w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) dot = fmaf(g[i] * w[i], n[i] * rstd, dot);
  }
  const float mean = block_sum(dot, sums) * p.inv_h;
  for (int c = threadIdx.x * kVec; c < p.H; c += step) {
    float g[kVec], n[kVec], w[kVec], o[kVec];
    load_vec<DT>(dy, c, p.H, g);
    load_vec<DT>(h, c, p.H, n);
    load_vec_dt(p.w, p.w_dt, c, p.H, w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) o[i] = rstd * (g[i] * w[i] - n[i] * rstd * mean);
    if (dh) {
      float u[kVec];
      load_vec<DT>(dh, c, p.H, u);
#pragma unroll
      for (int i = 0; i < kVec; ++i) o[i] += u[i];
    }
    store_vec(dx, DT, c, p.H, o);
  }
}

// dw: column sums of dy n.  A block owns 64 columns (8 lanes of one vector
// each) and walks all rows, 32 at a time; the 32 row groups' sums are added
// in order through shared memory.
template <int DT>
__global__ void __launch_bounds__(256)
rmsnorm_dw_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float part[32][64];
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int es = elem_bytes(DT);
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int c = blockIdx.x * 64 + lane * kVec;
  float acc[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
  if (c < p.H) {
    for (long long row = group; row < p.M; row += 32) {
      float g[kVec], n[kVec];
      load_vec<DT>(static_cast<const uint8_t*>(p.dy) + row * p.lddy * es, c, p.H, g);
      load_vec<DT>(static_cast<const uint8_t*>(p.h) + row * p.ldh * es, c, p.H, n);
      const float rstd = p.rstd[row];
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = fmaf(g[i], n[i] * rstd, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) part[group][lane * kVec + i] = acc[i];
  __syncthreads();
  const int col = blockIdx.x * 64 + (int)threadIdx.x;
  if (threadIdx.x < 64 && col < p.H) {
    float s = 0.f;
    for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
    store_elem(p.dw, col, p.dw_dt, s);
  }
}

}  // namespace gb300

namespace {

using namespace gb300host;

// Threads of a block that walks a row of H elements: a vector each, in whole
// warps, at most 1024.
int row_threads(int64_t H) {
  return (int)std::min<int64_t>(1024, cdiv(cdiv(H, gb300::kVec), 32) * 32);
}

gemm_status_t check_extents(int64_t M, int64_t H) {
  const int64_t kMax = INT32_MAX;
  if (M < 0 || H < 0 || M > kMax || H > kMax - 8192) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

gemm_status_t check_rmsnorm(const gemm_rmsnorm_t& p) {
  GB300_CHECK(check_extents(p.M, p.H));
  if (!is_epi_type(p.type) || !is_epi_type(p.w_type) || !(is_epi_type(p.y_type) || is_fp8(p.y_type)))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (p.M == 0 || p.H == 0) return GEMM_OK;
  GB300_CHECK(check_matrix(p.x, p.ldx, p.H, p.type));
  GB300_CHECK(check_matrix(p.y, p.ldy, p.H, p.y_type));
  if (p.r) GB300_CHECK(check_matrix(p.r, p.ldr, p.H, p.type));
  if (p.h) GB300_CHECK(check_matrix(p.h, p.ldh, p.H, p.type));
  if (!p.weight) return GEMM_ERR_INVALID_ARG;
  if (!aligned16(p.weight)) return GEMM_ERR_MISALIGNED;
  // an 8-bit output has a scale per row, and only it
  if (is_fp8(p.y_type) != (p.scale != nullptr)) return GEMM_ERR_INVALID_ARG;
  // in place: element for element only
  if (p.h && ((p.h == p.x && p.ldh != p.ldx) || (p.h == p.r && p.ldh != p.ldr)))
    return GEMM_ERR_INVALID_ARG;
  if ((p.y == p.x && (p.y_type != p.type || p.ldy != p.ldx)) ||
      (p.r && p.y == p.r && (p.y_type != p.type || p.ldy != p.ldr)) || (p.h && p.y == p.h))
    return GEMM_ERR_INVALID_ARG;
  if (!(p.eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

gemm_status_t check_rmsnorm_bwd(const gemm_rmsnorm_bwd_t& p) {
  GB300_CHECK(check_extents(p.M, p.H));
  if (!is_epi_type(p.type) || !is_epi_type(p.w_type) || !is_epi_type(p.dw_type))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (p.H == 0) return GEMM_OK;
  if (p.M > 0) {
    GB300_CHECK(check_matrix(p.dy, p.lddy, p.H, p.type));
    GB300_CHECK(check_matrix(p.h, p.ldh, p.H, p.type));
    GB300_CHECK(check_matrix(p.dx, p.lddx, p.H, p.type));
    if (p.dh) GB300_CHECK(check_matrix(p.dh, p.lddh, p.H, p.type));
    if (!p.weight || !p.rstd) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(p.weight)) return GEMM_ERR_MISALIGNED;
    if (p.dx == p.h || p.dx == p.dy || (p.dh && p.dx == p.dh && p.lddx != p.lddh))
      return GEMM_ERR_INVALID_ARG;
  }
  if (!p.dweight) return GEMM_ERR_INVALID_ARG;
  if (!aligned16(p.dweight)) return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

}  // namespace

GEMM_API gemm_status_t gemm_rmsnorm_check(const gemm_rmsnorm_t* p) {
  return p ? check_rmsnorm(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_rmsnorm_bwd_check(const gemm_rmsnorm_bwd_t* p) {
  return p ? check_rmsnorm_bwd(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_rmsnorm(gemm_handle_t h, const gemm_rmsnorm_t* pp,
                                    struct CUstream_st* stream) {
  NvtxRange range("gemm_rmsnorm");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_rmsnorm_t& p = *pp;
  GB300_CHECK(check_rmsnorm(p));
  if (p.M == 0 || p.H == 0) return GEMM_OK;
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  gb300::NormParams k{};
  k.x = p.x; k.ldx = p.ldx;
  k.r = p.r; k.ldr = p.ldr;
  k.h = p.h; k.ldh = p.ldh;
  k.w = p.weight; k.w_dt = device_dt(p.w_type);
  k.y = p.y; k.ldy = p.ldy; k.y_dt = device_dt(p.y_type);
  k.scale = p.scale;
  k.rstd = p.rstd;
  k.M = (int)p.M; k.H = (int)p.H;
  k.eps = p.eps;
  k.inv_h = (float)(1.0 / (double)p.H);
  void (*kern)(gb300::NormParams) = p.type == GEMM_F32   ? gb300::rmsnorm_any_kernel<gb300::DT_F32>
                                    : p.type == GEMM_F16 ? gb300::rmsnorm_any_kernel<gb300::DT_F16>
                                                         : gb300::rmsnorm_any_kernel<gb300::DT_BF16>;
  return launch(kern, k, p.M, row_threads(p.H), 0, stream);
}

GEMM_API int64_t gemm_rmsnorm_bwd_workspace(int64_t M, int64_t H) {
  (void)M; (void)H;
  return 0;
}

GEMM_API gemm_status_t gemm_rmsnorm_bwd(gemm_handle_t h, const gemm_rmsnorm_bwd_t* pp,
                                        void* workspace, int64_t workspace_bytes,
                                        struct CUstream_st* stream) {
  NvtxRange range("gemm_rmsnorm_bwd");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_rmsnorm_bwd_t& p = *pp;
  GB300_CHECK(check_rmsnorm_bwd(p));
  const int64_t need = gemm_rmsnorm_bwd_workspace(p.M, p.H);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GEMM_ERR_INVALID_ARG;
  if (need > 0 && !aligned16(workspace)) return GEMM_ERR_MISALIGNED;
  if (p.H == 0) return GEMM_OK;
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  gb300::NormBwdParams k{};
  k.dy = p.dy; k.lddy = p.lddy;
  k.h = p.h; k.ldh = p.ldh;
  k.w = p.weight; k.w_dt = device_dt(p.w_type);
  k.rstd = p.rstd;
  k.dh = p.dh; k.lddh = p.lddh;
  k.dx = p.dx; k.lddx = p.lddx;
  k.dw = p.dweight; k.dw_dt = device_dt(p.dw_type);
  k.M = (int)p.M; k.H = (int)p.H;
  k.inv_h = (float)(1.0 / (double)p.H);
  typedef void (*Kern)(gb300::NormBwdParams);
  Kern dx = p.type == GEMM_F32   ? gb300::rmsnorm_bwd_any_kernel<gb300::DT_F32>
            : p.type == GEMM_F16 ? gb300::rmsnorm_bwd_any_kernel<gb300::DT_F16>
                                 : gb300::rmsnorm_bwd_any_kernel<gb300::DT_BF16>;
  Kern dw = p.type == GEMM_F32   ? gb300::rmsnorm_dw_kernel<gb300::DT_F32>
            : p.type == GEMM_F16 ? gb300::rmsnorm_dw_kernel<gb300::DT_F16>
                                 : gb300::rmsnorm_dw_kernel<gb300::DT_BF16>;
  if (p.M > 0) GB300_CHECK(launch(dx, k, p.M, row_threads(p.H), 0, stream));
  return launch(dw, k, cdiv(p.H, 64), 256, 0, stream);
}
