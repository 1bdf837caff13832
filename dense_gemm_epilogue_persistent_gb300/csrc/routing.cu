// Tokens sorted by expert and back (include/gemm_gb300.h): the sort, the copy of the
// rows to their places, their weighted sum, and its gradients.
#include <algorithm>
#include <cstdint>

#include "gemm_gb300.h"
#include "handle.h"
#include "rows.cuh"
#include "rows_host.h"

namespace gb300 {

// ------------------------------------------------------------------ the sort

struct RouteParams {
  const void* index;
  long long ldi;
  int n, k, E;               // choices, choices of a token, experts
  int share;                 // choices of a warp: a multiple of 32
  int* offsets;
  int* slot;
  int* source;
};

constexpr int kRouteWarps = 32;
constexpr int kRouteCluster = 16;      // blocks, where the device takes so large a cluster; else 8
constexpr int kRouteAhead = 8;         // loads of 32 choices a warp has in flight

// A stable counting sort in one launch of one cluster (or one block).  Every warp
// owns a run of choices.  It counts them by expert, 32 at a time: lanes of one expert
// find one another by a vote on each of the BITS of its number, and one of them adds their
// number to the warp's counter, so that no two lanes ever add to one counter and no
// atomic decides an order; each choice's rank within the run is left in `slot`.  The
// counters, summed over warps, blocks (through distributed shared memory) and
// experts in that order, are the place of each warp's first choice of each expert, to
// which a second walk adds the ranks.  8 bytes a choice written, 8 to 16 read: the latency of
// the walks and sums, then the scattered stores of few SMs bound it.  (65536 choices of 64
// experts: 10.0 us; 13.5 by eight blocks, 14.1 so with the votes in both walks, 19.7 with match
// instructions there.)
template <typename T, int BITS>
__global__ void __launch_bounds__(32 * kRouteWarps)
route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int route_smem[];
  __shared__ int warp_sums[32];
  const int warps = (int)blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  int* const totals = route_smem;                // [E] choices of this block
  int* const before = totals + E;                // [E] first of this block's places, less ...
  int* const all = before + E;                   // [E] choices of the cluster
  int* const counts = all + E + warp * E;        // [E] ... this warp's
  const uint32_t blocks = gridDim.x, rank = blockIdx.x;    // (one cluster)
  grid_launch_dependents();
  for (int e = lane; e < E; e += 32) counts[e] = 0;
  __syncwarp();
  const long long first = min((long long)p.n, ((long long)rank * warps + warp) * p.share);
  const int count = (int)min((long long)p.share, p.n - first);
  grid_dependency_wait();

  const bool packed = p.ldi == p.k;
  const auto expert = [&](int i) {               // of the warp's i-th choice; -1: none
    if (i >= count) return -1;
    const long long c = first + i;
    const long long at = packed ? c : c / p.k * p.ldi + c % p.k;
    const T e = static_cast<const T*>(p.index)[at];
    return e >= 0 && e < (T)E ? (int)e : -1;
  };
  const auto walk = [&](auto&& f) {              // f(choice, expert) for 32 lanes at a time
    for (int i0 = 0; i0 < count; i0 += 32 * kRouteAhead) {
      int e[kRouteAhead];
#pragma unroll
      for (int u = 0; u < kRouteAhead; ++u) e[u] = expert(i0 + 32 * u + lane);
#pragma unroll
      for (int u = 0; u < kRouteAhead; ++u)
        if (i0 + 32 * u < count) f(i0 + 32 * u + lane, e[u]);
    }
  };
  walk([&](int i, int e) {
    // the lanes whose choice is this lane's (those without one among themselves)
    uint32_t same = __ballot_sync(0xFFFFFFFFu, e >= 0);
    if (e < 0) same = ~same;
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
      const bool one = e >> b & 1;
      const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one);
      same &= one ? ones : ~ones;
    }
    const uint32_t ahead = same & ((1u << lane) - 1u);
    const int so_far = e >= 0 ? counts[e] : 0;
    __syncwarp();
    if (e >= 0 && ahead == 0) counts[e] = so_far + __popc(same);
    __syncwarp();
    if (i < count) p.slot[first + i] = so_far + __popc(ahead);
  });
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < warps; ++w) {
      int* const c = all + E + w * E + e;
      const int mine = *c;
      *c = sum;
      sum += mine;
    }
    totals[e] = sum;
  }
  if (blocks > 1) cluster_sync_all(); else __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0, ahead = 0;
    if (blocks > 1) {
      for (uint32_t b = 0; b < blocks; ++b) {
        const int v = (int)load_cluster_u32(map_to_rank(smem_u32(totals + e), b));
        if (b < rank) ahead += v;
        sum += v;
      }
    } else {
      sum = totals[e];
    }
    all[e] = sum;
    before[e] = ahead;
  }
  __syncthreads();
  {
    // exclusive sums over the experts
    const int share = (E + (int)blockDim.x - 1) / (int)blockDim.x;
    const int e0 = min((int)threadIdx.x * share, E), e1 = min(e0 + share, E);
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += all[e];
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    int at = upto - mine, total = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) at += warp_sums[w];
      total += warp_sums[w];
    }
    for (int e = e0; e < e1; ++e) {
      if (rank == 0) p.offsets[e] = at;
      before[e] += at;
      at += all[e];
    }
    if (rank == 0 && threadIdx.x == 0) p.offsets[E] = total;
  }
  __syncthreads();
  for (int i0 = 0; i0 < count; i0 += 32 * kRouteAhead) {
    int e[kRouteAhead], rank[kRouteAhead];
#pragma unroll
    for (int u = 0; u < kRouteAhead; ++u) {
      const int i = i0 + 32 * u + lane;
      e[u] = expert(i);
      rank[u] = i < count ? p.slot[first + i] : 0;
    }
#pragma unroll
    for (int u = 0; u < kRouteAhead; ++u) {
      const int i = i0 + 32 * u + lane;
      const int place = e[u] >= 0 ? before[e[u]] + counts[e[u]] + rank[u] : -1;
      if (i < count) p.slot[first + i] = place;
      if (p.source && place >= 0) p.source[place] = (int)(first + i);
    }
  }
  if (blocks > 1) cluster_sync_all();            // the others have read this block's totals
}

// ------------------------------------------------------------------ the copy

struct DispatchParams {
  const uint8_t* x;
  uint8_t* y;
  long long ldx, ldy, row_bytes;     // bytes
  const int* slot;
  const float* scale;
  float* y_scale;
  long long T, R;
  int k, lanes, pieces;              // threads of a row; blocks that share it
};

constexpr int kCopyThreads = 128;
constexpr int kCopyVecs = 4;

// A token's row is read once, into registers, and stored at each of its choices' places:
// (1 + k) row bytes a token.  `lanes` threads a row (32 to 128), 4 pieces of 16 bytes
// each; longer rows are shared out to `pieces` blocks.
__global__ void __launch_bounds__(kCopyThreads)
dispatch_kernel(const __grid_constant__ DispatchParams p) {
  grid_launch_dependents();
  const int per_block = kCopyThreads / p.lanes;
  const long long t = (long long)(blockIdx.x / p.pieces) * per_block + threadIdx.x / p.lanes;
  const int piece = blockIdx.x % p.pieces, lane = threadIdx.x % p.lanes;
  grid_dependency_wait();
  if (t >= p.T) return;
  const uint8_t* const x = p.x + t * p.ldx;
  const long long c0 = ((long long)piece * kCopyVecs * p.lanes + lane) * 16;
  const long long step = (long long)p.lanes * 16;
  uint4 v[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i) {
    const long long c = c0 + i * step;
    if (c + 16 <= p.row_bytes) v[i] = __ldg(reinterpret_cast<const uint4*>(x + c));
  }
  const int* const slot = p.slot + t * p.k;
  const float scale = p.scale ? __ldg(p.scale + t) : 0.f;
#pragma unroll 4
  for (int j = 0; j < p.k; ++j) {
    const int s = __ldg(slot + j);
    if (s < 0 || s >= p.R) continue;
    uint8_t* const y = p.y + s * p.ldy;
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      const long long c = c0 + i * step;
      if (c + 16 <= p.row_bytes) {
        *reinterpret_cast<uint4*>(y + c) = v[i];
      } else {
        for (long long b = c; b < p.row_bytes; ++b) y[b] = x[b];    // the row's last bytes
      }
    }
    if (p.scale && piece == 0 && lane == 0) p.y_scale[s] = scale;
  }
}

// ------------------------------------------------------------------ the sum

struct CombineParams {
  const void* ys;
  const void* r;
  void* y;
  const int* slot;
  const float* weight;
  long long ldys, ldr, ldy;
  long long T, R;
  int k, H, lanes, pieces;
  int piece;                 // elements of a piece (the ring's)
  int r_dt, y_dt;
  uint32_t* status;          // (the ring's waits)
  unsigned long long timeout_ns;
};

constexpr int kSumThreads = 128;

// y = r + sum over the choices, fp32, in order.  `lanes` threads (32 to 128) a row, VECS vectors of 8
// columns each, ROWS rows' loads in flight; longer rows are cut into `pieces`, a block each.  For
// batches whose time is latency.
template <int DT, int VECS, int ROWS>
__global__ void __launch_bounds__(kSumThreads)
combine_kernel(const __grid_constant__ CombineParams p) {
  grid_launch_dependents();
  constexpr int es = elem_bytes(DT);
  const int per_block = kSumThreads / p.lanes;
  const long long t = (long long)(blockIdx.x / p.pieces) * per_block + threadIdx.x / p.lanes;
  const int piece = blockIdx.x % p.pieces, lane = threadIdx.x % p.lanes;
  grid_dependency_wait();
  if (t >= p.T) return;
  const int c0 = (piece * VECS * p.lanes + lane) * kVec, step = p.lanes * kVec;
  float acc[VECS][kVec];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[i][e] = 0.f;
    if (p.r && c0 + i * step < p.H)
      load_vec_dt(static_cast<const uint8_t*>(p.r) + t * p.ldr * elem_bytes(p.r_dt), p.r_dt,
                  c0 + i * step, p.H, acc[i]);
  }
  const int* const slot = p.slot + t * p.k;
  const float* const weight = p.weight ? p.weight + t * p.k : nullptr;
  for (int j0 = 0; j0 < p.k; j0 += ROWS) {
    int s[ROWS];
    float w[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      s[u] = j0 + u < p.k ? __ldg(slot + j0 + u) : -1;
      w[u] = weight && j0 + u < p.k ? __ldg(weight + j0 + u) : 1.f;
      if (s[u] >= p.R) s[u] = -1;
    }
    RawVec<DT> v[ROWS][VECS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const uint8_t* const row = static_cast<const uint8_t*>(p.ys) + (long long)s[u] * p.ldys * es;
#pragma unroll
      for (int i = 0; i < VECS; ++i)
        if (s[u] >= 0 && c0 + i * step < p.H) v[u][i] = load_raw<DT>(row, c0 + i * step, p.H);
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      if (s[u] < 0) continue;
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        if (c0 + i * step >= p.H) continue;
        float f[kVec];
        unpack<DT>(v[u][i], f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[i][e] = fmaf(w[u], f[e], acc[i][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VECS; ++i)
    if (c0 + i * step < p.H)
      store_vec(static_cast<uint8_t*>(p.y) + t * p.ldy * elem_bytes(p.y_dt), p.y_dt, c0 + i * step,
                p.H, acc[i]);
}

// The same for batches whose time is bandwidth.  A warp copies the choices' rows, pieces of up to 4 KB
// (bulk copies), into a ring of kRingSlots; kRingWarps warps add them up, VECS vectors of 8 columns
// a thread.  The copies run ahead of the sums by the whole ring, across tokens, and the
// places and weights by a token more, so that no wait for an address leaves memory idle.  A block takes
// about 700 cycles an entry, whatever its size, so that many small blocks an SM are wanted: 8192
// tokens of 8 x 4096 bf16 with a residual 104 us (6.5 TB/s; 116 with loads into registers), 112 with
// two blocks of twelve 8 KB slots; 4096 of 2 x 8192 42.5 (67.8), 61.8.
struct RingEntry {           // what a slot holds
  int row;                   // of ys; kResidual: the token's of r; -1: nothing (a token without choices)
  float weight;
  int flags;
};
constexpr int kResidual = -2;
enum : int { kLastEntry = 1, kWholeEntry = 2 };  // the token's last; its last 16 bytes are all there
constexpr int kRingSlots = 4, kRingWarps = 4, kRingBytes = 4096, kRingBlocks = 8;
constexpr int kRingThreads = 32 * (kRingWarps + 1);
constexpr int kRingSmem = kRingSlots * (kRingBytes + 16 + (int)sizeof(RingEntry)) + 16;

template <int DT, int VECS>
__global__ void __launch_bounds__(kRingThreads, kRingBlocks)
combine_ring_kernel(const __grid_constant__ CombineParams p) {
  constexpr int es = elem_bytes(DT);
  static_assert(32 * kRingWarps * VECS * kVec * es == kRingBytes, "a piece fills a slot");
  extern __shared__ __align__(16) uint8_t ring[];
  const uint32_t bars = smem_u32(ring) + kRingSlots * kRingBytes;
  RingEntry* const entries = reinterpret_cast<RingEntry*>(ring + kRingSlots * (kRingBytes + 16));
  volatile uint32_t* const abort_ptr = reinterpret_cast<volatile uint32_t*>(entries + kRingSlots);
  const auto full = [&](int s) { return bars + 16u * s; };
  const auto empty = [&](int s) { return bars + 16u * s + 8u; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRingSlots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kRingWarps);
    }
    *abort_ptr = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  const Watch w{abort_ptr, p.status, p.timeout_ns};
  // This block's piece of the rows (of p.piece elements, the last one shorter), and its tokens.
  const int piece = blockIdx.x % p.pieces;
  const int c_first = piece * p.piece, c_end = min(p.H, c_first + p.piece);
  // A residual of the rows' type comes through the ring too.
  const bool r_ring = p.r && p.r_dt == DT;
  const long long t_first = blockIdx.x / p.pieces, t_step = gridDim.x / p.pieces;
  int s = 0;
  uint32_t ph = 0;
  const auto advance = [&]() {
    if (++s == kRingSlots) { s = 0; ph ^= 1u; }
  };
  if (warp == kRingWarps) {
    // choices [j0, j0 + 32) of an item's token, one a lane; -1: none
    int row_next = -1;
    float w_next = 1.f;
    const auto look = [&](long long t, int j0) {
      const int j = j0 + lane;
      row_next = -1;
      w_next = 1.f;
      if (t < p.T && j < p.k) {
        const long long at = t * p.k + j;
        row_next = __ldg(p.slot + at);
        if (p.weight) w_next = __ldg(p.weight + at);
        if (row_next >= p.R) row_next = -1;
      }
    };
    bool ok = true;
    // One entry: a piece of a row, or none.
    const uint32_t bytes_here = (uint32_t)((c_end - c_first) * es);
    const auto push = [&](int row, float weight, bool last, long long t) {
      ok = __all_sync(0xFFFFFFFFu, wait_phase<true>(empty(s), ph ^ 1u, w, kWaitProducer));
      if (!ok) return;
      if (lane == 0) {
        // (Behind a matrix's last row there may be no more memory; behind another there is the next.)
        const bool whole = row == kResidual ? t + 1 < p.T : row + 1 < p.R;
        entries[s] = RingEntry{row, weight, (last ? kLastEntry : 0) | (whole ? kWholeEntry : 0)};
        const uint32_t bytes = row == -1 ? 0u : (whole ? bytes_here + 15u : bytes_here) & ~15u;
        mbar_arrive_expect_tx(full(s), bytes);
        if (bytes)
          bulk_load(smem_u32(ring) + s * kRingBytes,
                    (row == kResidual ? static_cast<const uint8_t*>(p.r) + t * p.ldr * es
                                      : static_cast<const uint8_t*>(p.ys) + (long long)row * p.ldys * es) +
                        (long long)c_first * es,
                    bytes, full(s));
      }
      __syncwarp();
      advance();
    };
    look(t_first, 0);
    for (long long t = t_first; ok && t < p.T; t += t_step) {
      // (an entry is pushed when the next is known, so that the last can be marked)
      int row = r_ring ? kResidual : -1;
      bool have = r_ring;
      float weight = 1.f;
      for (int j0 = 0; ok && j0 < p.k; j0 += 32) {
        const int row_now = row_next;
        const float w_now = w_next;
        if (j0 + 32 < p.k) look(t, j0 + 32);
        else look(t + t_step, 0);
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, row_now >= 0);
        for (uint32_t left = there; ok && left; left &= left - 1) {
          const int j = __ffs(left) - 1;
          if (have) push(row, weight, false, t);
          row = __shfl_sync(0xFFFFFFFFu, row_now, j);
          weight = __shfl_sync(0xFFFFFFFFu, w_now, j);
          have = true;
        }
      }
      if (ok) push(row, weight, true, t);
    }
  } else {
    const int c0 = c_first + (int)threadIdx.x * kVec;
    constexpr int step = 32 * kRingWarps * kVec;
    for (long long t = t_first; t < p.T; t += t_step) {
      float acc[VECS][kVec];
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[i][e] = 0.f;
        if (p.r && !r_ring && c0 + i * step < c_end)
          load_vec_dt(static_cast<const uint8_t*>(p.r) + t * p.ldr * elem_bytes(p.r_dt), p.r_dt,
                      c0 + i * step, p.H, acc[i]);
      }
      bool last = false;
      while (!last) {
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(full(s), ph, w, kWaitEpilogue))) break;
        const RingEntry entry = entries[s];
        last = entry.flags & kLastEntry;
        if (entry.row != -1) {
          const uint8_t* const slot = ring + s * kRingBytes;
          const uint8_t* const row =
              entry.row == kResidual ? static_cast<const uint8_t*>(p.r) + t * p.ldr * es
                                     : static_cast<const uint8_t*>(p.ys) + (long long)entry.row * p.ldys * es;
#pragma unroll
          for (int i = 0; i < VECS; ++i) {
            const int c = c0 + i * step;
            if (c >= c_end) continue;
            RawVec<DT> v;
            if (c + kVec <= p.H || (entry.flags & kWholeEntry)) {
              const uint4* const at = reinterpret_cast<const uint4*>(slot + (threadIdx.x * kVec + i * step) * es);
              v.q[0] = at[0];
              if constexpr (DT == DT_F32) v.q[1] = at[1];
            } else {
              v = load_raw<DT>(row, c, p.H);
            }
            float f[kVec];
            unpack<DT>(v, f);
#pragma unroll
            for (int e = 0; e < kVec; ++e) acc[i][e] = fmaf(entry.weight, f[e], acc[i][e]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(s));
        advance();
      }
      if (!last) break;                          // (a wait ran out)
#pragma unroll
      for (int i = 0; i < VECS; ++i)
        if (c0 + i * step < c_end)
          store_vec(static_cast<uint8_t*>(p.y) + t * p.ldy * elem_bytes(p.y_dt), p.y_dt,
                    c0 + i * step, p.H, acc[i]);
    }
  }
  __syncthreads();
  if (*abort_ptr) {
    // A wait gave up: let copies already issued drain first.
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
}

// ------------------------------------------------------------------ its gradients

struct CombineBwdParams {
  const void* dy;
  const void* ys;
  void* dys;
  const int* slot;
  const float* weight;
  float* dweight;
  long long lddy, ldys, lddys;
  long long R;
  int k, H;
};

constexpr int kBwdThreads = 256;       // at most
constexpr int kBwdVecs = 2;
constexpr int kBwdRows = 2;            // choices whose loads a thread has in flight
constexpr int kMaxChoices = 128;

// A block a token: its dy in registers, for each choice the row of dys and the product
// sum with the row of ys, two choices' loads in flight.  A choice's sum is added in a
// fixed order: a thread's columns, lanes, warps.  (1 + 2k) row bytes a token.
template <int DT>
__global__ void __launch_bounds__(kBwdThreads)
combine_bwd_kernel(const __grid_constant__ CombineBwdParams p) {
  __shared__ float part[kMaxChoices][kBwdThreads / 32];
  grid_launch_dependents();
  constexpr int es = elem_bytes(DT);
  const long long t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (int)blockDim.x >> 5;
  const int step = (int)blockDim.x * kVec;
  grid_dependency_wait();
  const uint8_t* const dy = static_cast<const uint8_t*>(p.dy) + t * p.lddy * es;
  const int* const slot = p.slot + t * p.k;
  const float* const weight = p.weight ? p.weight + t * p.k : nullptr;
  for (long long b = 0; b < p.H; b += (long long)step * kBwdVecs) {
    const int c0 = (int)b + threadIdx.x * kVec;
    float g[kBwdVecs][kVec];
#pragma unroll
    for (int i = 0; i < kBwdVecs; ++i) {
      if (c0 + i * step < p.H) {
        load_vec<DT>(dy, c0 + i * step, p.H, g[i]);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) g[i][e] = 0.f;
      }
    }
    for (int j0 = 0; j0 < p.k; j0 += kBwdRows) {
      int s[kBwdRows];
      RawVec<DT> v[kBwdRows][kBwdVecs];
#pragma unroll
      for (int u = 0; u < kBwdRows; ++u) {
        s[u] = j0 + u < p.k ? __ldg(slot + j0 + u) : -1;
        if (s[u] >= p.R) s[u] = -1;
        const uint8_t* const row = static_cast<const uint8_t*>(p.ys) + (long long)s[u] * p.ldys * es;
#pragma unroll
        for (int i = 0; i < kBwdVecs; ++i)
          if (p.dweight && s[u] >= 0 && c0 + i * step < p.H)
            v[u][i] = load_raw<DT>(row, c0 + i * step, p.H);
      }
#pragma unroll
      for (int u = 0; u < kBwdRows; ++u) {
        if (j0 + u >= p.k) break;
        float sum = 0.f;
        if (s[u] >= 0) {
          const float w = weight ? __ldg(weight + j0 + u) : 1.f;
          uint8_t* const out = static_cast<uint8_t*>(p.dys) + (long long)s[u] * p.lddys * es;
#pragma unroll
          for (int i = 0; i < kBwdVecs; ++i) {
            if (c0 + i * step >= p.H) continue;
            if (p.dweight) {
              float f[kVec];
              unpack<DT>(v[u][i], f);
#pragma unroll
              for (int e = 0; e < kVec; ++e) sum = fmaf(g[i][e], f[e], sum);
            }
            if (p.dys) {
              float o[kVec];
#pragma unroll
              for (int e = 0; e < kVec; ++e) o[e] = w * g[i][e];
              store_vec(out, DT, c0 + i * step, p.H, o);
            }
          }
        }
        if (p.dweight) {
          sum = warp_sum(sum);
          if (lane == 0) part[j0 + u][warp] = b ? part[j0 + u][warp] + sum : sum;
        }
      }
    }
  }
  if (!p.dweight) return;
  __syncthreads();
  for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
    float sum = 0.f;
    for (int w = 0; w < warps; ++w) sum += part[j][w];
    p.dweight[t * p.k + j] = sum;
  }
}

}  // namespace gb300

namespace {

using namespace gb300host;

// T tokens of k choices whose numbers fit 32 bits.
bool is_choices(int64_t T, int64_t k) {
  return is_extent(T) && k >= 0 && k <= gb300::kMaxChoices && is_extent(T * k);
}

gemm_status_t check_route(const gemm_route_t& p) {
  if (!is_choices(p.T, p.k) || p.E < 0 || p.E > 4096) return GEMM_ERR_INVALID_ARG;
  if (p.index_bytes != 4 && p.index_bytes != 8) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (!p.offsets) return GEMM_ERR_INVALID_ARG;
  if (!aligned_to(p.offsets, 4) || !aligned_to(p.slot, 4) || !aligned_to(p.source, 4) ||
      !aligned_to(p.index, p.index_bytes))
    return GEMM_ERR_MISALIGNED;
  if (p.T * p.k > 0 && (!p.index || !p.slot || p.ldi < p.k)) return GEMM_ERR_INVALID_ARG;
  if (p.T * p.k > 0 && (same_place(p.offsets, {p.index, p.slot, p.source}) ||
                        same_place(p.slot, {p.index, p.source}) || same_place(p.source, {p.index})))
    return GEMM_ERR_INVALID_ARG;       // (index is read again once slot has been written)
  return GEMM_OK;
}

// Places of the choices, and the R rows they are places of.
gemm_status_t check_places(int64_t T, int64_t k, int64_t H, int64_t R, const int32_t* slot) {
  if (!is_choices(T, k) || !is_extent(H) || !is_extent(R)) return GEMM_ERR_INVALID_ARG;
  if (T * k > 0 && !slot) return GEMM_ERR_INVALID_ARG;
  return aligned_to(slot, 4) ? GEMM_OK : GEMM_ERR_MISALIGNED;
}

gemm_status_t check_dispatch(const gemm_dispatch_t& p) {
  GB300_CHECK(check_places(p.T, p.k, p.H, p.R, p.slot));
  if (!is_epi_type(p.type) && !is_fp8(p.type)) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if ((p.scale != nullptr) != (p.y_scale != nullptr) || (p.scale && p.scale == p.y_scale))
    return GEMM_ERR_INVALID_ARG;
  if (!aligned_to(p.scale, 4) || !aligned_to(p.y_scale, 4)) return GEMM_ERR_MISALIGNED;
  if (p.T * p.k == 0 || p.R == 0) return GEMM_OK;
  if (same_place(p.y_scale, {p.slot})) return GEMM_ERR_INVALID_ARG;
  if (p.H == 0) return GEMM_OK;
  GB300_CHECK(check_matrix(p.x, p.ldx, p.H, p.type));
  GB300_CHECK(check_matrix(p.y, p.ldy, p.H, p.type));
  return same_place(p.y, {p.x, p.slot, p.scale, p.y_scale}) || same_place(p.y_scale, {p.x})
             ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

gemm_status_t check_combine(const gemm_combine_t& p) {
  GB300_CHECK(check_places(p.T, p.k, p.H, p.R, p.slot));
  if (!is_epi_type(p.type) || !is_epi_type(p.y_type) || (p.r && !is_epi_type(p.r_type)))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (!aligned_to(p.weight, 4)) return GEMM_ERR_MISALIGNED;
  if (p.T == 0 || p.H == 0) return GEMM_OK;
  GB300_CHECK(check_matrix(p.y, p.ldy, p.H, p.y_type));
  if (p.r) GB300_CHECK(check_matrix(p.r, p.ldr, p.H, p.r_type));
  if (p.k > 0 && p.R > 0) {
    GB300_CHECK(check_matrix(p.ys, p.ldys, p.H, p.type));
    if (same_place(p.y, {p.ys, p.slot, p.weight})) return GEMM_ERR_INVALID_ARG;
  }
  if (p.r == p.y && (p.r_type != p.y_type || p.ldr != p.ldy)) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

gemm_status_t check_combine_bwd(const gemm_combine_bwd_t& p) {
  GB300_CHECK(check_places(p.T, p.k, p.H, p.R, p.slot));
  if (!is_epi_type(p.type)) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (!aligned_to(p.weight, 4) || !aligned_to(p.dweight, 4)) return GEMM_ERR_MISALIGNED;
  if (p.T * p.k == 0) return GEMM_OK;
  if (same_place(p.dweight, {p.weight, p.slot})) return GEMM_ERR_INVALID_ARG;
  if (p.H == 0 || p.R == 0) return GEMM_OK;
  GB300_CHECK(check_matrix(p.dy, p.lddy, p.H, p.type));
  if (p.dweight) GB300_CHECK(check_matrix(p.ys, p.ldys, p.H, p.type));
  if (same_place(p.dweight, {p.dy, p.ys})) return GEMM_ERR_INVALID_ARG;
  if (p.dys) {
    GB300_CHECK(check_matrix(p.dys, p.lddys, p.H, p.type));
    if (same_place(p.dys, {p.dy, p.slot, p.weight, p.dweight}) || (p.dweight && p.dys == p.ys && p.lddys != p.ldys))
      return GEMM_ERR_INVALID_ARG;
  }
  return GEMM_OK;
}

template <typename T>
void (*route_kernel(int bits))(gb300::RouteParams) {
  return bits <= 3   ? gb300::route_kernel<T, 3>
         : bits <= 6 ? gb300::route_kernel<T, 6>
         : bits <= 8 ? gb300::route_kernel<T, 8>
                     : gb300::route_kernel<T, 12>;
}

// Blocks of the sort's cluster (h->mu held): 16, which a kernel has to be allowed first, if one with as much
// shared memory as any call asks for fits the device; else 8.
gemm_status_t route_cluster(gemm_handle* h, void (*kern)(gb300::RouteParams), size_t smem, int* blocks) {
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (h->route_cluster == 0) {
    int n = 0;
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute attr[1];
    lc.gridDim = dim3((unsigned)gb300::kRouteCluster);
    lc.blockDim = dim3(32 * gb300::kRouteWarps);
    lc.dynamicSmemBytes = smem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)gb300::kRouteCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &lc) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    h->route_cluster = n > 0 ? gb300::kRouteCluster : 8;
  }
  *blocks = h->route_cluster;
  return GEMM_OK;
}

// Threads of a row (32, 64 or 128) that take `vecs` of its `total` vectors each.
int row_lanes(int64_t total, int vecs) {
  int lanes = 32;
  while (lanes < 128 && (int64_t)lanes * vecs < total) lanes *= 2;
  return lanes;
}

}  // namespace

GEMM_API gemm_status_t gemm_route_check(const gemm_route_t* p) {
  return p ? check_route(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_route(gemm_handle_t h, const gemm_route_t* pp,
                                  struct CUstream_st* stream) {
  NvtxRange range("gemm_route");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_route_t& p = *pp;
  GB300_CHECK(check_route(p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  gb300::RouteParams k{};
  k.index = p.index; k.ldi = p.ldi;
  k.n = (int)(p.T * p.k); k.k = (int)std::max<int64_t>(1, p.k); k.E = (int)p.E;
  k.offsets = p.offsets; k.slot = p.slot; k.source = p.source;
  // As many warps as their counters leave room for; up to 2048 choices one block, whose
  // warps take 32 choices or more each.
  const int room = (h->smem_optin - 2048) / 4;
  const int fit = p.E > 0 ? (int)std::min<int64_t>(gb300::kRouteWarps, (room - 3 * p.E) / p.E)
                          : gb300::kRouteWarps;
  int bits = 0;
  while ((1ll << bits) < p.E) ++bits;
  typedef void (*Kern)(gb300::RouteParams);
  const Kern kern = p.index_bytes == 8 ? route_kernel<long long>(bits) : route_kernel<int>(bits);
  int blocks = 1;
  {
    std::lock_guard<std::mutex> guard(h->mu);
    GB300_CHECK(raise_smem(h, reinterpret_cast<const void*>(kern)));
    if (k.n > 2048) GB300_CHECK(route_cluster(h, kern, (size_t)room * 4, &blocks));
  }
  const int warps = blocks > 1 ? fit : std::min(fit, std::max(4, (int)cdiv(k.n, 32)));
  k.share = (int)cdiv(cdiv(k.n, (int64_t)blocks * warps), 32) * 32;
  const size_t smem = (size_t)(3 + warps) * p.E * 4;
  return launch(kern, k, blocks, 32 * warps, smem, stream, blocks);
}

GEMM_API gemm_status_t gemm_dispatch_check(const gemm_dispatch_t* p) {
  return p ? check_dispatch(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_dispatch(gemm_handle_t h, const gemm_dispatch_t* pp,
                                     struct CUstream_st* stream) {
  NvtxRange range("gemm_dispatch");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_dispatch_t& p = *pp;
  GB300_CHECK(check_dispatch(p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  if (p.T * p.k == 0 || p.R == 0 || (p.H == 0 && !p.scale)) return GEMM_OK;
  const int es = dtype_bytes(p.type);
  gb300::DispatchParams k{};
  k.x = static_cast<const uint8_t*>(p.x); k.ldx = p.ldx * es;
  k.y = static_cast<uint8_t*>(p.y); k.ldy = p.ldy * es;
  k.row_bytes = p.H * es;
  k.slot = p.slot;
  k.scale = p.scale; k.y_scale = p.y_scale;
  k.T = p.T; k.R = p.R;
  k.k = (int)p.k;
  const int64_t vecs = std::max<int64_t>(1, cdiv(k.row_bytes, 16));
  k.lanes = row_lanes(vecs, gb300::kCopyVecs);
  k.pieces = (int)cdiv(vecs, (int64_t)k.lanes * gb300::kCopyVecs);
  const int64_t grid = cdiv(p.T, gb300::kCopyThreads / k.lanes) * k.pieces;
  if (grid > INT32_MAX) return GEMM_ERR_INVALID_ARG;
  return launch(gb300::dispatch_kernel, k, grid, gb300::kCopyThreads, 0, stream);
}

GEMM_API gemm_status_t gemm_combine_check(const gemm_combine_t* p) {
  return p ? check_combine(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_combine(gemm_handle_t h, const gemm_combine_t* pp,
                                    struct CUstream_st* stream) {
  NvtxRange range("gemm_combine");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_combine_t& p = *pp;
  GB300_CHECK(check_combine(p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  if (p.T == 0 || p.H == 0) return GEMM_OK;
  gb300::CombineParams k{};
  k.ys = p.ys; k.ldys = p.ldys;
  k.r = p.r; k.ldr = p.ldr; k.r_dt = device_dt(p.r_type);
  k.y = p.y; k.ldy = p.ldy; k.y_dt = device_dt(p.y_type);
  k.slot = p.slot; k.weight = p.weight;
  k.T = p.T; k.R = p.R;
  k.k = (int)p.k; k.H = (int)p.H;
  typedef void (*Kern)(gb300::CombineParams);
  const int es = dtype_bytes(p.type);
  // The ring from 4 KB a row and 32 MB on (8192 tokens of 8 x 512 bf16 36.6 us by the ring, 18.0
  // without; 1024 of 8 x 4096 17.3, 17.7; 512 of 8 x 4096 9.5, 10.5).
  if (p.H * es >= 4096 && (double)p.T * (double)p.k * (double)p.H * es >= 32e6) {
    k.pieces = (int)cdiv(p.H, gb300::kRingBytes / es);
    k.piece = (int)cdiv(cdiv(p.H, k.pieces), gb300::kVec) * gb300::kVec;
    k.status = h->d_status;
    k.timeout_ns = h->timeout_ns;
    const Kern kern = p.type == GEMM_F32   ? (Kern)gb300::combine_ring_kernel<gb300::DT_F32, 1>
                      : p.type == GEMM_F16 ? (Kern)gb300::combine_ring_kernel<gb300::DT_F16, 2>
                                           : (Kern)gb300::combine_ring_kernel<gb300::DT_BF16, 2>;
    {
      std::lock_guard<std::mutex> guard(h->mu);
      GB300_CHECK(raise_smem(h, reinterpret_cast<const void*>(kern)));
    }
    const int64_t blocks = std::max<int64_t>(1, gb300::kRingBlocks * h->sm_count / k.pieces);    // of a piece
    return launch(kern, k, std::min(p.T, blocks) * k.pieces, gb300::kRingThreads, gb300::kRingSmem,
                  stream);
  }
  const int64_t vecs = cdiv(p.H, gb300::kVec);
  k.lanes = row_lanes(vecs, 2);
  k.pieces = (int)cdiv(vecs, (int64_t)k.lanes * 2);
  const int64_t grid = cdiv(p.T, gb300::kSumThreads / k.lanes) * k.pieces;
  if (grid > INT32_MAX) return GEMM_ERR_INVALID_ARG;
  const Kern kern = p.type == GEMM_F32   ? (Kern)gb300::combine_kernel<gb300::DT_F32, 2, 2>
                    : p.type == GEMM_F16 ? (Kern)gb300::combine_kernel<gb300::DT_F16, 2, 4>
                                         : (Kern)gb300::combine_kernel<gb300::DT_BF16, 2, 4>;
  return launch(kern, k, grid, gb300::kSumThreads, 0, stream);
}

GEMM_API gemm_status_t gemm_combine_bwd_check(const gemm_combine_bwd_t* p) {
  return p ? check_combine_bwd(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_combine_bwd(gemm_handle_t h, const gemm_combine_bwd_t* pp,
                                        struct CUstream_st* stream) {
  NvtxRange range("gemm_combine_bwd");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_combine_bwd_t& p = *pp;
  GB300_CHECK(check_combine_bwd(p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  if (p.T * p.k == 0 || (!p.dys && !p.dweight)) return GEMM_OK;
  gb300::CombineBwdParams k{};
  k.dy = p.dy; k.lddy = p.lddy;
  k.ys = p.ys; k.ldys = p.ldys;
  k.dys = p.dys; k.lddys = p.lddys;
  k.slot = p.slot; k.weight = p.weight; k.dweight = p.dweight;
  k.R = p.R;
  k.k = (int)p.k; k.H = (int)p.H;
  if (p.H == 0 || p.R == 0) {
    // no row to read or write: every choice's weight has gradient 0
    if (!p.dweight) return GEMM_OK;
    if (cudaMemsetAsync(p.dweight, 0, (size_t)(p.T * p.k) * 4,
                        reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
  }
  const int64_t vecs = cdiv(p.H, gb300::kVec);
  // as few passes over the row as there can be, of one length
  const int64_t passes = cdiv(vecs, (int64_t)gb300::kBwdThreads * gb300::kBwdVecs);
  const int threads = (int)(cdiv(cdiv(vecs, gb300::kBwdVecs * passes), 32) * 32);
  typedef void (*Kern)(gb300::CombineBwdParams);
  const Kern kern = p.type == GEMM_F32   ? (Kern)gb300::combine_bwd_kernel<gb300::DT_F32>
                    : p.type == GEMM_F16 ? (Kern)gb300::combine_bwd_kernel<gb300::DT_F16>
                                         : (Kern)gb300::combine_bwd_kernel<gb300::DT_BF16>;
  return launch(kern, k, p.T, threads, 0, stream);
}
