// Low-rank adapters of few rows (a decode batch, short prompts among it): one kernel without matrix
// units.  A cluster of blocks has the rows of a request, or up to 16 clusters have every 16th of them: each block the sums over its share of
// the inner size, which the cluster adds up through distributed shared memory, then its share of
// the features.  The bytes of a row's adapter are asked for at once, those of the second matrix
// before the first sums, so that what bounds a call are a memory latency or two a wave of blocks
// and the launch; of a request with many rows one row after the other, which is where products over groups of rows take
// over.  (64 requests of a row, rank 16, 4096 x 4096 bf16: 8.0 us, the host's call included, 7.0 in a graph; 41.8 by
// products, each tile of which moves and multiplies 128 features for its one row; 10.3 by two kernels, one
// a matrix.)
#pragma once

#include "rows.cuh"

namespace gb300 {

struct FewParams {
  int M, N, K, rank, requests, adapters;
  int splits;                // clusters that share a request's rows
  const int* offsets;
  const int* index;
  const void* x; long long ldx;
  const void* a; long long lda, stride_a;
  const void* b; long long ldb, stride_b;
  const float* scale;
  const void* r; long long ldr;
  void* d; long long ldd;
  int r_dt, d_dt, in_place;
};

constexpr int kFewThreads = 256;
constexpr int kFewCluster = 8;
constexpr int kFewPer = 2;             // ranks of a warp at a time
constexpr int kFewAhead = 2;           // ... and vectors of each that a lane has in flight
constexpr int kFewRank = 1024;         // ranks at most (shared memory)

// Rows [first, last) of request s, clamped to the matrix; its adapter, or -1.
__device__ __forceinline__ int few_request(const FewParams& p, int s, int& first, int& last) {
  first = min(max(__ldg(p.offsets + s), 0), p.M);
  last = min(max(__ldg(p.offsets + s + 1), 0), p.M);
  const int e = __ldg(p.index + s);
  return e >= 0 && e < p.adapters ? e : -1;
}

// u(m, j) = sum_k x(m, k) A(e, j, k): a warp has ranks, its lanes every 32nd vector of the block's
// share; partial sums are added in the order lanes, blocks, and stay fp32: u never leaves shared
// memory, so nothing is saved by rounding it to DT as the products' workspace has it.
// d(m, n) = r(m, n) + scale(e) sum_j u(m, j) B(e, n, j): LANES lanes read a row of B together (8 ranks
// each: up to 128 contiguous bytes), in LANES passes over a warp's 32 features; then every
// lane takes over the sums of one of the features of its LANES (a lane that keeps a half of its
// sums gives the other half away, LANES / 2, ..., 1 at a time) and has feature `lane` of the 32.
template <int DT, int LANES>
__global__ void __launch_bounds__(kFewThreads)
adapters_few_kernel(const __grid_constant__ FewParams p) {
  __shared__ float parts[2][kFewRank];           // this block's sums, of even and odd rows
  __shared__ float us[kFewRank];
  constexpr int es = elem_bytes(DT);
  constexpr int kWarps = kFewThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x % kFewCluster, split = blockIdx.x / kFewCluster % p.splits;
  const int s = blockIdx.x / kFewCluster / p.splits;
  const int part = threadIdx.x % LANES;
  grid_launch_dependents();
  grid_dependency_wait();
  int first, last;
  const int e = few_request(p, s, first, last);
  first += split;
  if (first >= last || (e < 0 && p.in_place)) return;          // (the whole cluster)
  const uint8_t* const a = static_cast<const uint8_t*>(p.a) + max(e, 0) * p.stride_a * es;
  const uint8_t* const b = static_cast<const uint8_t*>(p.b) + max(e, 0) * p.stride_b * es;
  const int share = ((p.K + kVec - 1) / kVec + kFewCluster - 1) / kFewCluster;
  const int k_first = block * share * kVec, k_last = min(p.K, k_first + share * kVec);
  const int chunks = (p.N + kFewThreads - 1) / kFewThreads;     // of features: every kFewCluster-th is the block's
  // the vector of ranks j .. j + 7 of the feature of pass i of a chunk
  const auto load = [&](int chunk, int i, int j) {
    const int n = chunk * kFewThreads + (int)threadIdx.x - part + i;
    RawVec<DT> raw{};
    if (chunk < chunks && n < p.N && j < p.rank) raw = load_raw<DT>(b + (long long)n * p.ldb * es, j, p.rank);
    return raw;
  };
  const auto residual = [&](int m, int chunk) {
    const int n = chunk * kFewThreads + threadIdx.x;
    return p.r && chunk < chunks && n < p.N ? load_elem_dt(p.r, (long long)m * p.ldr + n, p.r_dt) : 0.f;
  };
  RawVec<DT> raw[LANES];
  float scale = 1.f;
  if (e >= 0) {
    if (p.scale) scale = __ldg(p.scale + e);
#pragma unroll
    for (int i = 0; i < LANES; ++i) raw[i] = load(block, i, part * kVec);
  }
  int turn = 0;
#pragma unroll 1
  for (int m = first; m < last; m += p.splits, turn ^= 1) {
    float res = residual(m, block);
    if (e >= 0) {
      const uint8_t* const x = static_cast<const uint8_t*>(p.x) + (long long)m * p.ldx * es;
#pragma unroll 1
      for (int j = warp * kFewPer; j < p.rank; j += kWarps * kFewPer) {
        float acc[kFewPer] = {};
#pragma unroll 1
        for (int k0 = k_first + lane * kVec; k0 < k_last; k0 += kFewAhead * 32 * kVec) {
          RawVec<DT> av[kFewPer][kFewAhead], xv[kFewAhead];
#pragma unroll
          for (int i = 0; i < kFewAhead; ++i) {
            const int k = k0 + i * (32 * kVec);
#pragma unroll
            for (int c = 0; c < kFewPer; ++c) {
              av[c][i] = RawVec<DT>{};
              if (k < k_last && j + c < p.rank) av[c][i] = load_raw<DT>(a + (long long)(j + c) * p.lda * es, k, p.K);
            }
            xv[i] = RawVec<DT>{};
            if (k < k_last) xv[i] = load_raw<DT>(x, k, p.K);
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
          if (lane == 0 && j + c < p.rank) parts[turn][j + c] = sum;
        }
      }
      // (the sums of a row are read while the next row's are made; those of the one after next are not
      // before all blocks have read them)
      cluster_sync_all();
      for (int j = threadIdx.x; j < (p.rank + kVec - 1) / kVec * kVec; j += kFewThreads) {
        float sum = 0.f;
        if (j < p.rank) {
#pragma unroll
          for (uint32_t c = 0; c < kFewCluster; ++c)
            sum += __uint_as_float(load_cluster_u32(map_to_rank(smem_u32(&parts[turn][j]), c)));
        }
        us[j] = sum;
      }
      __syncthreads();
    }
    for (int chunk = block; chunk < chunks; chunk += kFewCluster) {
      float acc[LANES] = {};
      const float here = res;
      res = residual(m, chunk + kFewCluster);
#pragma unroll 1
      for (int j = part * kVec; e >= 0 && j < p.rank; j += LANES * kVec) {
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
        // the next vectors: of these features, of the next chunk, or the first again for the next row
        const bool more = j + LANES * kVec < p.rank;
        const int then = more ? chunk : chunk + kFewCluster < chunks ? chunk + kFewCluster : block;
#pragma unroll
        for (int i = 0; i < LANES; ++i) raw[i] = load(then, i, more ? j + LANES * kVec : part * kVec);
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
      const int n = chunk * kFewThreads + threadIdx.x;
      if (n < p.N) store_elem(p.d, (long long)m * p.ldd + n, p.d_dt, fmaf(scale, acc[0], here));
    }
    __syncthreads();                             // (us has been read)
  }
  if (e >= 0) cluster_sync_all();                // the others have read this block's sums
}

}  // namespace gb300
