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

// A row held in registers: read once, written once.  T threads (a block, or a
// warp where WARP: then a block holds 4 rows) keep VPT vectors of the row each,
// vector i of thread t being elements 8 (i T + t).  The outputs follow two
// reductions over the row (sum of squares; largest output magnitude where the
// output is 8-bit).  DRAM-bound: 4 es + eo bytes an element with a residual.
template <int DT, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024)
rmsnorm_row_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[32];
  __shared__ uint32_t maxs[32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int T = WARP ? 32 : blockDim.x;
  const long long row = WARP ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.M) return;
  constexpr int es = elem_bytes(DT);
  const uint8_t* const x = static_cast<const uint8_t*>(p.x) + row * p.ldx * es;
  RawVec<DT> xv[VPT], rv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * T + t) * kVec;
    if (c < p.H) xv[i] = load_raw<DT>(x, c, p.H);
    else xv[i] = RawVec<DT>{};
  }
  if (p.r) {
    const uint8_t* const r = static_cast<const uint8_t*>(p.r) + row * p.ldr * es;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
      if (c < p.H) rv[i] = load_raw<DT>(r, c, p.H);
      else rv[i] = RawVec<DT>{};
    }
  }
  float v[VPT][kVec];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    unpack<DT>(xv[i], v[i]);
    if (p.r) {
      float u[kVec];
      unpack<DT>(rv[i], u);
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[i][k] += u[k];
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k) ss = fmaf(v[i][k], v[i][k], ss);
  }
  const float total = WARP ? warp_sum(ss) : block_sum(ss, sums);
  const float rstd = 1.f / sqrtf(total * p.inv_h + p.eps);
  if (t == 0 && p.rstd) p.rstd[row] = rstd;
  if (p.h) {
    uint8_t* const h = static_cast<uint8_t*>(p.h) + row * p.ldh * es;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
      if (c < p.H) store_vec(h, DT, c, p.H, v[i]);
    }
  }
  const bool fp8 = p.y_dt >= DT_E4M3;
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * T + t) * kVec;
    if (c >= p.H) continue;
    float w[kVec];
    load_vec_dt(p.w, p.w_dt, c, p.H, w);
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      v[i][k] = v[i][k] * rstd * w[k];
      big = max(big, abs_bits(v[i][k]));
    }
  }
  float inv = 1.f;
  if (fp8) {
    big = WARP ? __reduce_max_sync(0xFFFFFFFFu, big) : block_max(big, maxs);
    big = max(big, __float_as_uint(kAmaxFloor));
    const float amax = __uint_as_float(big), top = largest_fp8(p.y_dt);
    inv = top / amax;
    if (t == 0) p.scale[row] = amax / top;
  }
  uint8_t* const y = static_cast<uint8_t*>(p.y) + row * p.ldy * elem_bytes(p.y_dt);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * T + t) * kVec;
    if (c >= p.H) continue;
    if (fp8) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[i][k] *= inv;
    }
    store_vec(y, p.y_dt, c, p.H, v[i]);
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
  float* partials;                  // rows of H partial weight gradients
};

struct SumParams {
  const float* partials;
  void* out;
  int rows, H, out_dt;
};

// Partial sums [c, c + 8) of a row of H floats (rows of any alignment).
__device__ __forceinline__ void store_partial(float* row, int c, int n, const float (&v)[kVec]) {
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (c + k < n) row[c + k] = v[k];
}

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

// Both gradients in one reading of dy, h and dh.  Blocks walk the rows
// blockIdx.x, + gridDim.x, ...; each thread keeps the same VPT vectors of
// columns throughout (a block's T threads span a row; with WARP a warp does and
// the block's 8 warps take different rows), so the weight gradient of the rows
// it has seen stays in its registers.  The next row's vectors are requested
// before the current row's reduction.  At the end every block writes its H
// sums to the workspace; sum_partials_kernel adds them in block order.
template <int DT, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512)
rmsnorm_bwd_row_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float sums[2][32];
  extern __shared__ float warp_dw[];     // WARP: 8 rows of H sums
  grid_launch_dependents();
  grid_dependency_wait();
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int T = WARP ? 32 : blockDim.x;
  const int walkers = WARP ? gridDim.x * 8 : gridDim.x;
  constexpr int es = elem_bytes(DT);
  RawVec<DT> g_raw[VPT], h_raw[VPT], d_raw[VPT];
  auto fetch = [&](long long row) {
    const uint8_t* const dy = static_cast<const uint8_t*>(p.dy) + row * p.lddy * es;
    const uint8_t* const h = static_cast<const uint8_t*>(p.h) + row * p.ldh * es;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
      if (c >= p.H) continue;
      g_raw[i] = load_raw<DT>(dy, c, p.H);
      h_raw[i] = load_raw<DT>(h, c, p.H);
      if (p.dh)
        d_raw[i] = load_raw<DT>(static_cast<const uint8_t*>(p.dh) + row * p.lddh * es, c, p.H);
    }
  };
  float dw[VPT][kVec];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    g_raw[i] = h_raw[i] = d_raw[i] = RawVec<DT>{};
#pragma unroll
    for (int k = 0; k < kVec; ++k) dw[i][k] = 0.f;
  }
  const int first = WARP ? (int)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (first < p.M) fetch(first);
  int buf = 0;
  for (long long row = first; row < p.M; row += walkers, buf ^= 1) {
    float n[VPT][kVec], g[VPT][kVec], u[VPT][kVec];
    const float rstd = p.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack<DT>(g_raw[i], g[i]);
      unpack<DT>(h_raw[i], n[i]);
      unpack<DT>(d_raw[i], u[i]);
    }
    if (row + walkers < p.M) fetch(row + walkers);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
      float w[kVec];
      if (c < p.H) {
        load_vec_dt(p.w, p.w_dt, c, p.H, w);
      } else {
#pragma unroll
        for (int k = 0; k < kVec; ++k) w[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        n[i][k] *= rstd;
        dw[i][k] = fmaf(g[i][k], n[i][k], dw[i][k]);
        g[i][k] *= w[k];
        dot = fmaf(g[i][k], n[i][k], dot);
      }
    }
    const float mean = (WARP ? warp_sum(dot) : block_sum(dot, sums[buf])) * p.inv_h;
    uint8_t* const dx = static_cast<uint8_t*>(p.dx) + row * p.lddx * es;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
      if (c >= p.H) continue;
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        g[i][k] = rstd * (g[i][k] - n[i][k] * mean);
        if (p.dh) g[i][k] += u[i][k];
      }
      store_vec(dx, DT, c, p.H, g[i]);
    }
  }
  float* const out = p.partials + (long long)blockIdx.x * p.H;
  if constexpr (!WARP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
      if (c < p.H) store_partial(out, c, p.H, dw[i]);
    }
  } else {
    float* const mine = warp_dw + (threadIdx.x >> 5) * p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (c + k < p.H) mine[c + k] = dw[i][k];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.H; c += 256) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += warp_dw[k * p.H + c];
      out[c] = s;
    }
  }
}

// Column sums of `rows` rows of H partial sums: 32 columns a block, 32 row
// groups, added in order.
__global__ void __launch_bounds__(1024)
sum_partials_kernel(const __grid_constant__ SumParams p) {
  __shared__ float part[32][33];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < p.H) {
#pragma unroll 4
    for (int r = group; r < p.rows; r += 32) s += p.partials[(long long)r * p.H + c];
  }
  part[group][lane] = s;
  __syncthreads();
  if (group == 0 && c < p.H) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][lane];
    store_elem(p.out, c, p.out_dt, s);
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

// Rows up to kRowMax elements are held in registers: vectors per thread and
// threads per row (a warp's 32 where warp).
constexpr int kRowMax = 32768, kBwdRowMax = 16384;
struct RowShape {
  int vpt, threads;
  bool warp;
};

RowShape forward_shape(int64_t M, int64_t H) {
  const int vecs = (int)cdiv(H, gb300::kVec);
  (void)M;
  RowShape s{};
  if (vecs <= 128) {
    s.warp = true;
    s.vpt = vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4;
    s.threads = 128;
    return s;
  }
  s.vpt = vecs <= 256 ? 1 : vecs <= 2048 ? 2 : 4;
  s.threads = (int)cdiv(cdiv(vecs, s.vpt), 32) * 32;
  return s;
}

RowShape backward_shape(int64_t H) {
  const int vecs = (int)cdiv(H, gb300::kVec);
  RowShape s{};
  if (vecs <= 128) {
    s.warp = true;
    s.vpt = vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4;
    s.threads = 256;
    return s;
  }
  s.vpt = vecs <= 256 ? 1 : vecs <= 1024 ? 2 : 4;
  s.threads = (int)cdiv(cdiv(vecs, s.vpt), 32) * 32;
  return s;
}

// Blocks of the backward row kernel (one row of partial sums each).
constexpr int kBwdBlocks = 304;
int backward_blocks(int64_t M, int64_t H) {
  const RowShape s = backward_shape(H);
  return (int)std::min<int64_t>(s.warp ? cdiv(M, 8) : M, kBwdBlocks);
}

typedef void (*NormKern)(gb300::NormParams);
template <int DT, bool WARP>
NormKern forward_kernel(int vpt) {
  return vpt == 1   ? gb300::rmsnorm_row_kernel<DT, 1, WARP>
         : vpt == 2 ? gb300::rmsnorm_row_kernel<DT, 2, WARP>
                    : gb300::rmsnorm_row_kernel<DT, 4, WARP>;
}
template <int DT>
NormKern forward_kernel(const RowShape& s) {
  return s.warp ? forward_kernel<DT, true>(s.vpt) : forward_kernel<DT, false>(s.vpt);
}

typedef void (*NormBwdKern)(gb300::NormBwdParams);
template <int DT, bool WARP>
NormBwdKern backward_kernel(int vpt) {
  return vpt == 1   ? gb300::rmsnorm_bwd_row_kernel<DT, 1, WARP>
         : vpt == 2 ? gb300::rmsnorm_bwd_row_kernel<DT, 2, WARP>
                    : gb300::rmsnorm_bwd_row_kernel<DT, 4, WARP>;
}
template <int DT>
NormBwdKern backward_kernel(const RowShape& s) {
  return s.warp ? backward_kernel<DT, true>(s.vpt) : backward_kernel<DT, false>(s.vpt);
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
  if (p.H <= kRowMax) {
    const RowShape s = forward_shape(p.M, p.H);
    return launch(p.type == GEMM_F32   ? forward_kernel<gb300::DT_F32>(s)
                  : p.type == GEMM_F16 ? forward_kernel<gb300::DT_F16>(s)
                                       : forward_kernel<gb300::DT_BF16>(s),
                  k, s.warp ? cdiv(p.M, 4) : p.M, s.threads, 0, stream);
  }
  NormKern kern = p.type == GEMM_F32   ? gb300::rmsnorm_any_kernel<gb300::DT_F32>
                                    : p.type == GEMM_F16 ? gb300::rmsnorm_any_kernel<gb300::DT_F16>
                                                         : gb300::rmsnorm_any_kernel<gb300::DT_BF16>;
  return launch(kern, k, p.M, row_threads(p.H), 0, stream);
}

GEMM_API int64_t gemm_rmsnorm_bwd_workspace(int64_t M, int64_t H) {
  if (M <= 0 || H <= 0 || H > kBwdRowMax) return 0;
  return backward_blocks(M, H) * H * (int64_t)sizeof(float);
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
  if (need > 0) {
    const RowShape s = backward_shape(p.H);
    const int blocks = backward_blocks(p.M, p.H);
    k.partials = static_cast<float*>(workspace);
    GB300_CHECK(launch(p.type == GEMM_F32   ? backward_kernel<gb300::DT_F32>(s)
                       : p.type == GEMM_F16 ? backward_kernel<gb300::DT_F16>(s)
                                            : backward_kernel<gb300::DT_BF16>(s),
                       k, blocks, s.threads, s.warp ? 8 * (size_t)p.H * sizeof(float) : 0, stream));
    gb300::SumParams q{k.partials, p.dweight, blocks, (int)p.H, k.dw_dt};
    return launch(gb300::sum_partials_kernel, q, cdiv(p.H, 32), 1024, 0, stream);
  }
  NormBwdKern dx = p.type == GEMM_F32   ? gb300::rmsnorm_bwd_any_kernel<gb300::DT_F32>
            : p.type == GEMM_F16 ? gb300::rmsnorm_bwd_any_kernel<gb300::DT_F16>
                                 : gb300::rmsnorm_bwd_any_kernel<gb300::DT_BF16>;
  NormBwdKern dw = p.type == GEMM_F32   ? gb300::rmsnorm_dw_kernel<gb300::DT_F32>
            : p.type == GEMM_F16 ? gb300::rmsnorm_dw_kernel<gb300::DT_F16>
                                 : gb300::rmsnorm_dw_kernel<gb300::DT_BF16>;
  if (p.M > 0) GB300_CHECK(launch(dx, k, p.M, row_threads(p.H), 0, stream));
  return launch(dw, k, cdiv(p.H, 64), 256, 0, stream);
}
