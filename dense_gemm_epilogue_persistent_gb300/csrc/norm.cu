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
// output is 8-bit).  DRAM-bound: 3 es + eo bytes an element with a residual and h (es, eo the
// types' sizes), es + eo without.
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
  int depth;                        // rows a thread requests ahead
};

struct SumParams {
  const float* partials;
  void* out;
  int rows, H, ld, out_dt;
};

// Floats from one row of partial sums to the next: whole 16-byte pieces.
__host__ __device__ constexpr int partial_ld(int H) { return (H + 3) & ~3; }

// The backward kernel's blocks stay and walk rows first, first + walkers, ...;
// every thread copies its own vectors of the next rows into its own slots of
// shared memory with cp.async, `depth` rows ahead, so no thread waits on
// another for data and the loads in flight do not depend on registers or on the
// reductions.  cp.async's byte count clips the row's end exactly (the rest of
// the 16 bytes reads as zero).

// A thread's slots for one vector of each of its rows: 16-byte pieces of one
// tensor lie blockDim.x pieces apart, so a warp's pieces are contiguous.
template <int DT, int VPT>
struct RowPipe {
  static constexpr int kPieces = DT == DT_F32 ? 2 : 1;      // 16-byte pieces of a vector
  static constexpr int kPer = VPT * kPieces;                // ... of a thread's row of one tensor
  // Request this thread's part of a row into slot `s` (tensor slots).
  __device__ static __forceinline__ void request(uint8_t* smem, int s, const uint8_t* row, int t,
                                                 int T, int H) {
    constexpr int es = elem_bytes(DT);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int c = (i * T + t) * kVec + k * (16 / es);
        const int bytes = min(16, max(0, (H - c) * es));
        const uint8_t* const src = bytes > 0 ? row + (size_t)c * es : row;
        copy16_async(smem_u32(smem + ((size_t)(s * kPer + i * kPieces + k) * blockDim.x +
                                      threadIdx.x) * 16),
                     src, bytes);
      }
    }
  }
  __device__ static __forceinline__ void read(const uint8_t* smem, int s, int i, float (&v)[kVec]) {
    RawVec<DT> raw;
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      raw.q[k] = *reinterpret_cast<const uint4*>(
          smem + ((size_t)(s * kPer + i * kPieces + k) * blockDim.x + threadIdx.x) * 16);
    unpack<DT>(raw, v);
  }
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

// Both gradients in one reading of dy, h and dh, requested ahead through RowPipe.
// Each thread keeps the same VPT vectors of columns throughout (a block's threads
// span a row; with WARP a warp does and the block's 8 warps take different rows), so
// the weight gradient of the rows it has seen stays in its registers.  At the end
// every block writes its H sums to the workspace; sum_partials_kernel adds them in a
// fixed order.
template <int DT, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512)
rmsnorm_bwd_rows_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float sums[2][32];
  extern __shared__ __align__(16) uint8_t slots[];     // afterwards, WARP: 8 rows of H sums
  using Pipe = RowPipe<DT, VPT>;
  grid_launch_dependents();
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int T = WARP ? 32 : blockDim.x;
  const int walkers = WARP ? gridDim.x * 8 : gridDim.x;
  const int first = WARP ? (int)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  constexpr int es = elem_bytes(DT);
  const int D = p.depth, tensors = p.dh ? 3 : 2;
  grid_dependency_wait();
  auto request = [&](long long row, int s) {
    if (row < p.M) {
      const int q = s * tensors;
      Pipe::request(slots, q, static_cast<const uint8_t*>(p.dy) + row * p.lddy * es, t, T, p.H);
      Pipe::request(slots, q + 1, static_cast<const uint8_t*>(p.h) + row * p.ldh * es, t, T, p.H);
      if (p.dh)
        Pipe::request(slots, q + 2, static_cast<const uint8_t*>(p.dh) + row * p.lddh * es, t, T,
                      p.H);
    }
    copy_commit();
  };
  for (int s = 0; s < D; ++s) request(first + (long long)s * walkers, s);
  float dw[VPT][kVec], w[VPT][kVec];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * T + t) * kVec;
#pragma unroll
    for (int k = 0; k < kVec; ++k) dw[i][k] = w[i][k] = 0.f;
    if (c < p.H) load_vec_dt(p.w, p.w_dt, c, p.H, w[i]);
  }
  float next_rstd = first < p.M ? p.rstd[first] : 0.f;
  int s = 0, buf = 0;
  for (long long row = first; row < p.M; row += walkers, buf ^= 1) {
    const float rstd = next_rstd;
    if (row + walkers < p.M) next_rstd = p.rstd[row + walkers];
    copy_wait(D - 1);
    float n[VPT][kVec], g[VPT][kVec];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      Pipe::read(slots, s * tensors, i, g[i]);
      Pipe::read(slots, s * tensors + 1, i, n[i]);
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        n[i][k] *= rstd;
        dw[i][k] = fmaf(g[i][k], n[i][k], dw[i][k]);
        g[i][k] *= w[i][k];
        dot = fmaf(g[i][k], n[i][k], dot);
      }
    }
    const float mean = (WARP ? warp_sum(dot) : block_sum(dot, sums[buf])) * p.inv_h;
    uint8_t* const dx = static_cast<uint8_t*>(p.dx) + row * p.lddx * es;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
#pragma unroll
      for (int k = 0; k < kVec; ++k) g[i][k] = rstd * (g[i][k] - n[i][k] * mean);
      if (p.dh) {
        float u[kVec];
        Pipe::read(slots, s * tensors + 2, i, u);
#pragma unroll
        for (int k = 0; k < kVec; ++k) g[i][k] += u[k];
      }
      if (c < p.H) store_vec(dx, DT, c, p.H, g[i]);
    }
    request(row + (long long)D * walkers, s);
    if (++s == D) s = 0;
  }
  copy_wait(0);
  float* const out = p.partials + (long long)blockIdx.x * partial_ld(p.H);
  if constexpr (!WARP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * T + t) * kVec;
      if (c < p.H) store_vec(out, DT_F32, c, p.H, dw[i]);
    }
  } else {
    float* const warp_dw = reinterpret_cast<float*>(slots);
    float* const mine = warp_dw + (threadIdx.x >> 5) * p.H;
    __syncthreads();                     // the slots are free
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

// Column sums of `rows` rows of partial sums, `ld` floats apart: a warp's lanes
// take 4 columns each, a block's 32 warps rows w, w + 32, ..., added in that
// order and then in warp order.
__global__ void __launch_bounds__(1024)
sum_partials_kernel(const __grid_constant__ SumParams p) {
  __shared__ float4 part[32][32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < p.H) {
#pragma unroll 10
    for (int r = group; r < p.rows; r += 32) {
      const float4 v = *reinterpret_cast<const float4*>(p.partials + (long long)r * p.ld + c);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  part[group][lane] = s;
  __syncthreads();
  if (threadIdx.x < 128) {
    const int col = blockIdx.x * 128 + (int)threadIdx.x;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += reinterpret_cast<const float*>(part[i])[threadIdx.x];
    if (col < p.H) store_elem(p.out, col, p.out_dt, t);
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

// Forward rows up to kRowMax elements are held in registers, a warp's up to
// 1024 elements and a block's above: vectors per thread and threads.
constexpr int kRowMax = 32768, kBwdRowMax = 16384;
struct RowShape {
  int vpt, threads;
  bool warp;
};

// One, two or four vectors a thread, by an estimate of each: up to two waves of
// blocks, waves x (1.5 us + the bytes of a full wave's rows), beyond that all bytes at
// the rate each reaches (90, 80, 60 % of 6.8 TB/s).  Fewer threads a row leave more
// rows in flight, and DRAM busier (8192 x 8192 bf16 -> E4M3 with residual: 73.9 us at
// 4 vectors, 94.1 at 2, 118 at 1); more threads a row shorten it where its latency or
// a last wave counts (1000 x 5003: 11.2 us at 2, 13.0 at 4; 600 x 2048: 3.4 at 1, 4.7 at
// 4), up to 768 of them, where their joining costs more again (1 x 8192: 3.09 us at 2,
// 3.33 at 1, 3.73 at 4).  Over 178 sizes (1 to 7000 rows of 1536 to 12000) the choice is
// 1.1 % over the fastest on average, 12 % at worst.  (Fitted on 16-bit rows; 32-bit ones
// take the same rates, and their four-vector block kernel spills 104 bytes a thread.)
RowShape forward_shape(int64_t M, int64_t H, int64_t row_bytes, int sm_count) {
  const int vecs = (int)cdiv(H, gb300::kVec);
  RowShape s{};
  s.warp = vecs <= 128;
  if (s.warp) {
    s.vpt = vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4;
    s.threads = 128;
    return s;
  }
  double best = 0.0;
  for (int v : {1, 2, 4}) {
    const int threads = (int)cdiv(cdiv(vecs, v), 32) * 32;
    if (threads > 768 && v < 4) continue;
    const int regs = v == 4 ? 64 : v == 2 ? 48 : 32;     // as compiled, in allocation steps
    const int64_t slots =
        (int64_t)sm_count * std::max(1, std::min(2048 / threads, 65536 / (regs * threads)));
    const int64_t waves = cdiv(M, slots);
    const double rate = v == 4 ? 0.9 : v == 2 ? 0.8 : 0.6;
    const double us =
        waves <= 2 ? (double)waves * (1.5 + (double)(std::min(M, slots) * row_bytes) / 6.8e6)
                   : 1.5 + (double)M * (double)row_bytes / (6.8e6 * rate);
    if (s.vpt == 0 || us < best) {
      best = us;
      s.vpt = v;
      s.threads = threads;
    }
  }
  return s;
}

// The backward row kernel: two vectors a thread and about 512 threads an SM
// (their registers fill it), two rows ahead: 8192 x 8192 bf16 with dh 87.4 us
// at 2 vectors x 512 threads x 2 rows against 105 with 4 x 256 x 1 and 122 with
// 1 block of each; 32768 x 2048: 84.8 us with 4 blocks of 128 threads, 89.7 with
// 8, 100.8 with 1 vector.  Longer rows (over 8192) take 4 vectors, one row ahead
// (4096 x 16384: 112 us, 121 with two), and spill 68 bytes a thread, 104 in 32 bits.
struct BwdShape {
  int vpt, threads, blocks_per_sm, depth;
  bool warp;
};

BwdShape backward_shape(int64_t H) {
  const int vecs = (int)cdiv(H, gb300::kVec);
  BwdShape s{};
  s.warp = vecs <= 128;
  if (s.warp) {
    s.vpt = vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4;
    s.threads = 256;
    s.blocks_per_sm = s.vpt == 4 ? 1 : 2;
  } else {
    s.vpt = vecs <= 1024 ? 2 : 4;
    s.threads = (int)cdiv(cdiv(vecs, s.vpt), 32) * 32;
    s.blocks_per_sm = std::max(1, 512 / s.threads);
  }
  // (4-byte rows of four vectors a thread: two do not fit in shared memory)
  s.depth = s.vpt == 4 && !s.warp ? 1 : 2;
  return s;
}

// Most blocks the backward row kernel runs on (one row of partial sums each):
// its blocks per SM on 152 SMs, as many as leave a block three rows (partial sums
// are written and read again: 600 x 2048 8.9 us with one block an SM, 10.9 with four).
int backward_blocks(int64_t M, int64_t H) {
  const BwdShape s = backward_shape(H);
  const int64_t per_sm = s.warp ? s.blocks_per_sm
                                : std::max<int64_t>(1, std::min<int64_t>(s.blocks_per_sm, M / 456));
  return (int)std::min<int64_t>(s.warp ? cdiv(M, 8) : M, 152 * per_sm);
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
  if constexpr (WARP)                            // (a block's threads take two or four)
    if (vpt == 1) return gb300::rmsnorm_bwd_rows_kernel<DT, 1, WARP>;
  return vpt == 2 ? gb300::rmsnorm_bwd_rows_kernel<DT, 2, WARP>
                  : gb300::rmsnorm_bwd_rows_kernel<DT, 4, WARP>;
}
template <int DT>
NormBwdKern backward_kernel(const BwdShape& s) {
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
  if (!aligned_to(p.scale, 4) || !aligned_to(p.rstd, 4)) return GEMM_ERR_MISALIGNED;
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
    if (!aligned16(p.weight) || !aligned_to(p.rstd, 4)) return GEMM_ERR_MISALIGNED;
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
    const int64_t row_bytes = p.H * (dtype_bytes(p.type) * (1 + (p.r != nullptr) + (p.h != nullptr)) +
                                     dtype_bytes(p.y_type));
    const RowShape s = forward_shape(p.M, p.H, row_bytes, h->sm_count);
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
  return backward_blocks(M, H) * (int64_t)gb300::partial_ld((int)H) * (int64_t)sizeof(float);
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
    const BwdShape s = backward_shape(p.H);
    const int blocks = (int)std::min<int64_t>(backward_blocks(p.M, p.H),
                                              (int64_t)h->sm_count * s.blocks_per_sm);
    k.partials = static_cast<float*>(workspace);
    k.depth = s.depth;
    NormBwdKern kern = p.type == GEMM_F32   ? backward_kernel<gb300::DT_F32>(s)
                       : p.type == GEMM_F16 ? backward_kernel<gb300::DT_F16>(s)
                                            : backward_kernel<gb300::DT_BF16>(s);
    {
      std::lock_guard<std::mutex> guard(h->mu);
      GB300_CHECK(raise_smem(h, reinterpret_cast<const void*>(kern)));
    }
    const size_t slots = (size_t)s.depth * (p.dh ? 3 : 2) * s.threads * s.vpt * gb300::kVec *
                         dtype_bytes(p.type);
    const size_t sums = s.warp ? 8 * (size_t)p.H * sizeof(float) : 0;
    GB300_CHECK(launch(kern, k, blocks, s.threads, std::max(slots, sums), stream));
    gb300::SumParams q{k.partials, p.dweight, blocks, k.H, gb300::partial_ld(k.H), k.dw_dt};
    return launch(gb300::sum_partials_kernel, q, cdiv(p.H, 128), 1024, 0, stream);
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
