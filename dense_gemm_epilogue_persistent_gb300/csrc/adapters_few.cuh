// Low-rank adapters of requests with a row or two each (a decode batch): two kernels without
// matrix units.  Every byte of a row's adapter is asked for at once, the second kernel's
// before the first has ended, so that what bounds a call are two memory latencies a
// wave of blocks and the launch.  (64 requests of a row, rank 16, 4096 x 4096 bf16: 10.3 us, the host's call included; 36.2 by
// products over groups of rows, each tile of which moves and multiplies 128 features for
// its one row.)
#pragma once

#include "rows.cuh"

namespace gb300 {

struct FewParams {
  int M, N, K, rank, requests, adapters;
  int chunks, splits;        // blocks of a request: ranks (down) or features (up), rows
  const int* offsets;
  const int* index;
  const void* x; long long ldx;
  const void* a; long long lda, stride_a;
  const void* b; long long ldb, stride_b;
  const float* scale;
  void* u; long long ldu;
  const void* r; long long ldr;
  void* d; long long ldd;
  int r_dt, d_dt, in_place;
};

constexpr int kFewThreads = 256;
constexpr int kFewParts = 2;           // warps that share a rank's inner products
constexpr int kFewPer = 2;             // ranks of a warp
constexpr int kFewRanks = kFewThreads / 32 / kFewParts * kFewPer;    // ranks of a block
constexpr int kFewAhead = 4;           // vectors of a rank that a lane has in flight
constexpr int kFewU = 256;             // ranks whose u is held in shared memory at a time

// Rows [first, last) of request s, clamped to the matrix; its adapter, or -1.
__device__ __forceinline__ int few_request(const FewParams& p, int s, int& first, int& last) {
  first = min(max(__ldg(p.offsets + s), 0), p.M);
  last = min(max(__ldg(p.offsets + s + 1), 0), p.M);
  const int e = __ldg(p.index + s);
  return e >= 0 && e < p.adapters ? e : -1;
}

// u(m, j) = sum_k x(m, k) A(e, j, k): kFewParts warps take kFewPer ranks, each every kFewParts-th vector
// of a lane, partial sums added in that order.
template <int DT>
__global__ void __launch_bounds__(kFewThreads)
adapters_down_kernel(const __grid_constant__ FewParams p) {
  __shared__ float sums[kFewPer][kFewThreads / 32];
  constexpr int es = elem_bytes(DT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % p.splits, chunk = blockIdx.x / p.splits % p.chunks;
  const int s = blockIdx.x / p.splits / p.chunks;
  grid_dependency_wait();
  // (only now: what the next kernel reads before its own wait is then complete)
  grid_launch_dependents();
  int first, last;
  const int e = few_request(p, s, first, last);
  if (e < 0) return;
  const int j = chunk * kFewRanks + warp / kFewParts * kFewPer, part = warp % kFewParts;
  const uint8_t* const a = static_cast<const uint8_t*>(p.a) + e * p.stride_a * es;
#pragma unroll 1
  for (int m = first + split; m < last; m += p.splits) {
    const uint8_t* const x = static_cast<const uint8_t*>(p.x) + (long long)m * p.ldx * es;
    float acc[kFewPer] = {};
#pragma unroll 1
    for (int k0 = (part * 32 + lane) * kVec; k0 < p.K; k0 += kFewAhead * kFewParts * 32 * kVec) {
      RawVec<DT> av[kFewPer][kFewAhead], xv[kFewAhead];
#pragma unroll
      for (int i = 0; i < kFewAhead; ++i) {
        const int k = k0 + i * (kFewParts * 32 * kVec);
#pragma unroll
        for (int c = 0; c < kFewPer; ++c) {
          av[c][i] = RawVec<DT>{};
          if (k < p.K && j + c < p.rank) av[c][i] = load_raw<DT>(a + (long long)(j + c) * p.lda * es, k, p.K);
        }
        xv[i] = RawVec<DT>{};
        if (k < p.K) xv[i] = load_raw<DT>(x, k, p.K);
      }
#pragma unroll
      for (int i = 0; i < kFewAhead; ++i) {
        float g[kVec];
        unpack<DT>(xv[i], g);
#pragma unroll
        for (int c = 0; c < kFewPer; ++c) {
          float f[kVec];
          unpack<DT>(av[c][i], f);
#pragma unroll
          for (int v = 0; v < kVec; ++v) acc[c] = fmaf(f[v], g[v], acc[c]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kFewPer; ++c) {
      const float sum = warp_sum(acc[c]);
      if (lane == 0) sums[c][warp] = sum;
    }
    __syncthreads();
    if (part == 0 && lane < kFewPer && j + lane < p.rank) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) sum += sums[lane][warp + i];
      store_elem(p.u, (long long)m * p.ldu + j + lane, DT, sum);
    }
    __syncthreads();
  }
}

// d(m, n) = r(m, n) + scale(e) sum_j u(m, j) B(e, n, j).  LANES lanes read a row of B together (8 ranks
// each: up to 128 contiguous bytes), in LANES passes over a warp's 32 features; then every
// lane takes over the sums of one of the features of its LANES (a lane that keeps a half of its
// sums gives the other half away, LANES / 2, ..., 1 at a time) and has feature `lane` of the 32.
template <int DT, int LANES>
__global__ void __launch_bounds__(kFewThreads)
adapters_up_kernel(const __grid_constant__ FewParams p) {
  __shared__ float us[kFewU];
  constexpr int es = elem_bytes(DT);
  const int split = blockIdx.x % p.splits, chunk = blockIdx.x / p.splits % p.chunks;
  const int s = blockIdx.x / p.splits / p.chunks;
  const int n = chunk * kFewThreads + threadIdx.x;             // the feature in the end
  const int part = threadIdx.x % LANES, n_first = n - part;    // ... and the first of its LANES
  grid_launch_dependents();
  // The first kernel lets this one start after its own wait: all that ran before it is complete, and
  // it writes u only.
  int first, last;
  const int e = few_request(p, s, first, last);
  first += split;
  const bool any = first < last && (e >= 0 || !p.in_place);
  const uint8_t* const b = static_cast<const uint8_t*>(p.b) + max(e, 0) * p.stride_b * es;
  // the vector of ranks j .. j + 7 of the feature of pass i
  const auto load = [&](int i, int j) {
    RawVec<DT> raw{};
    if (n_first + i < p.N && j < p.rank)
      raw = load_raw<DT>(b + (long long)(n_first + i) * p.ldb * es, j, p.rank);
    return raw;
  };
  RawVec<DT> raw[LANES];
  float scale = 1.f;
  if (any && e >= 0) {
    if (p.scale) scale = __ldg(p.scale + e);
#pragma unroll
    for (int i = 0; i < LANES; ++i) raw[i] = load(i, part * kVec);
  }
  grid_dependency_wait();
  if (!any) return;
#pragma unroll 1
  for (int m = first; m < last; m += p.splits) {
    const float res =
        p.r && n < p.N ? load_elem_dt(p.r, (long long)m * p.ldr + n, p.r_dt) : 0.f;
    float acc[LANES] = {};
    for (int j0 = 0; e >= 0 && j0 < p.rank; j0 += kFewU) {
      const int ranks = min(kFewU, p.rank - j0);
      __syncthreads();
      for (int j = threadIdx.x; j < (ranks + kVec - 1) / kVec * kVec; j += kFewThreads)
        us[j] = j < ranks ? load_elem<DT>(p.u, (long long)m * p.ldu + j0 + j) : 0.f;
      __syncthreads();
#pragma unroll 1
      for (int j = part * kVec; j < ranks; j += LANES * kVec) {
        float g[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) g[v] = us[j + v];
#pragma unroll
        for (int i = 0; i < LANES; ++i) {
          float f[kVec];
          unpack<DT>(raw[i], f);
#pragma unroll
          for (int v = 0; v < kVec; ++v) acc[i] = fmaf(g[v], f[v], acc[i]);
        }
        // the next vectors: of this row, or the first again for the next one
        const int next = j0 + j + LANES * kVec;
#pragma unroll
        for (int i = 0; i < LANES; ++i) raw[i] = load(i, next < p.rank ? next : part * kVec);
      }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      const bool high = part & o;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float give = high ? acc[i] : acc[i + o], keep = high ? acc[i + o] : acc[i];
        acc[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
      }
    }
    if (n < p.N) store_elem(p.d, (long long)m * p.ldd + n, p.d_dt, fmaf(scale, acc[0], res));
  }
}

}  // namespace gb300
