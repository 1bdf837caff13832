// Products over groups of rows, each group with weights of its own (sm_103a):
//
//   rows     z[m,n] = alpha scale[e] row_scale[m] col_scale[e,n] sum_k a[m,k] b[e,n,k] + bias[e,n]
//            d = act(z) + r   for the rows m of group g, e = index[g] (g without an index)
//   weights  d[g,c,f] = alpha sum_m dz[m,c] a[m,f] (+ d)   over the rows m of group g
//
// Group g's rows are offsets[g] .. offsets[g + 1] - 1 of the token matrix, in device
// memory: the host knows neither their number nor their place, so every CTA builds
// the list of work items itself (a prefix sum over the groups in shared memory)
// and walks it with the others, item by item in turn.
//
// The features lie on the MMA's rows (tensor-memory lanes), the tokens on its
// columns.  A tile's width then follows its group in steps of 16 or 64 columns, so
// that a ragged group costs no more than its own rows; an accumulator column is
// one token, whose 32 features a warp stores as one contiguous piece; nothing is
// ever written between the groups, whatever lies next to them, and neither row
// ends nor tile ends need padding.  (Rows of other groups inside a token box give
// columns that are not stored.)
//
// In the weights form the group's rows are the inner dimension.  Its last block
// runs as many 16-row MMA steps as hold rows; where the last of them holds others',
// a warp of its own zeroes those rows of both operands in shared memory
// before the MMA (a product with zeros in one operand only would keep another
// group's infinities).  The two CTAs of a pair do so each for its own half: such a
// stage's copies report to a barrier of the CTA, and the zeroing warps' arrivals
// complete the stage.
//
// Block: warp 0 TMA producer, warp 1 tensor memory and MMA issue, warps 2-9
// epilogue (two per lane quarter, taking 16-column chunks alternately), warp 10 (weights
// form) the zeroing.  Persistent grid of CTAs or CTA pairs, one CTA an SM, two
// accumulator stages.  Bound by the tensor pipe for large groups, by the
// weights' DRAM traffic for small ones.  The waits are bounded as in gemm_kernel.cuh.
#pragma once

#include "activations.cuh"
#include "gemm_kernel.cuh"

namespace gb300 {

struct GroupedParams {
  int rows;                  // of the token matrix: groups are clamped to them
  int feats;                 // output features (MMA rows)
  int cols;                  // weights form: output rows of a group (MMA columns)
  int k;                     // rows form: inner size
  int groups, sets;          // groups of rows, sets of weights
  int bn;                    // widest tile
  int unit;                  // columns of one box of the token operand
  int tiles_f, tiles_c;      // feature tiles; weights form: column tiles
  int stages;
  int f_mn;                  // rows form: weights with contiguous features
  int has_operands;          // the tensor maps are encoded
  int skip_none;             // groups without weights are left out: their d is r already
  uint32_t idesc;            // instruction descriptor without the tile width
  const int* offsets;        // [groups + 1]
  const int* index;          // [groups], or null
  uint32_t* status;
  unsigned long long timeout_ns;
  int inject_stall;
  // epilogue
  float alpha;
  const float* set_scale;    // [sets], or null
  const float* row_scale;    // [rows], or null
  const float* col_scale;    // [sets, feats], or null
  const void* bias;          // [sets, feats], or null
  const void* r;             // residual (the weights form's own d where it is added to), or null
  void* z;                   // or null
  void* d;
  long long ldr, ldz, ldd;   // row strides, elements
  long long sd;              // weights form: a group's stride, of d and r
  int bias_dt, r_dt, z_dt, d_dt, act;
};

constexpr int kGroupedKA = 2;                  // 128-byte K atoms a ring stage
constexpr int kGroupedEpiWarps = 8;
constexpr int kGroupedChunk = 16;              // columns of an epilogue chunk
constexpr int kGroupedStrip = 8;               // token tiles walked together for L2
constexpr int kGroupedMaxGroups = 4096;        // what the tables in shared memory hold
constexpr int kGroupedMaxStages = 8;

constexpr int grouped_threads(bool weights) { return 64 + 32 * kGroupedEpiWarps + (weights ? 32 : 0); }

// Bytes of a ring stage and of what follows the ring: barriers (full, empty, tail; two
// accumulators' full and empty; one that nothing arrives at), tensor-memory
// address and abort flag, warps' sums, the two tables.
constexpr int grouped_stage_bytes(int cta_group, int bn) {
  return kGroupedKA * (128 + bn / cta_group) * 128;
}
constexpr int grouped_bar_bytes() { return 8 * (3 * kGroupedMaxStages + 5) + 16 + 64; }
constexpr int grouped_smem(int cta_group, int bn, int stages, int groups) {
  return 1024 + stages * grouped_stage_bytes(cta_group, bn) + grouped_bar_bytes() + 8 * (groups + 1);
}

__device__ __forceinline__ uint32_t grouped_elem(const uint8_t* p, int dt) {
  return dt == DT_F32 ? *reinterpret_cast<const uint32_t*>(p)
                      : (uint32_t)*reinterpret_cast<const uint16_t*>(p);
}

// 16 values, `count` of them, `step` bytes apart.
__device__ __forceinline__ void grouped_store(uint8_t* p, long long step, int dt, int count,
                                              const float (&v)[kGroupedChunk]) {
  if (dt == DT_F32) {
#pragma unroll
    for (int i = 0; i < kGroupedChunk; ++i)
      if (i < count) *reinterpret_cast<float*>(p + i * step) = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < kGroupedChunk; i += 2) {
      const uint32_t w = dt == DT_F16 ? pack_f16x2(v[i], v[i + 1]) : pack_bf16x2(v[i], v[i + 1]);
      if (i < count) *reinterpret_cast<uint16_t*>(p + i * step) = (uint16_t)w;
      if (i + 1 < count) *reinterpret_cast<uint16_t*>(p + (i + 1) * step) = (uint16_t)(w >> 16);
    }
  }
}

template <int CG, int AB_BYTES, bool kWeights>
__global__ void __launch_bounds__(grouped_threads(kWeights), 1)
grouped_kernel(const __grid_constant__ CUtensorMap tmF, const __grid_constant__ CUtensorMap tmT,
               const __grid_constant__ GroupedParams p) {
  constexpr int KIND = (AB_BYTES == 1) ? 1 : (AB_BYTES == 4 ? 2 : 0);
  constexpr int KA = kGroupedKA;
  constexpr int ATOM_K = 128 / AB_BYTES;         // K of a 128-byte atom; features of an MN-major one
  constexpr int BK = ATOM_K * KA;                // inner size of a stage
  constexpr int UMMA_K = 32 / AB_BYTES;
  constexpr int K_STEPS = BK / UMMA_K;
  constexpr int STEPS_PER_ATOM = ATOM_K / UMMA_K;
  constexpr uint32_t MN_ATOM = BK * 128;         // bytes of an MN-major atom column
  constexpr uint32_t F_ATOM = 128 * 128;         // bytes of a K-major atom of 128 features
  constexpr uint32_t F_STAGE = F_ATOM * KA;
  constexpr int F_BOXES = 128 / ATOM_K;          // MN-major boxes of the 128 features
  constexpr bool PAIR = CG == 2;
  static_assert(!kWeights || AB_BYTES == 2, "weight gradients are of 16-bit operands");

  grid_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // the same in both CTAs of a pair
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int cluster_id = blockIdx.x / CG, num_clusters = gridDim.x / CG;
  const int S = p.stages, bn = p.bn;
  const uint32_t t_atom = (uint32_t)(bn / CG) * 128u;    // K-major atom of the CTA's tokens
  const uint32_t t_stage = t_atom * KA;
  const uint32_t f_ring = base, t_ring = f_ring + S * F_STAGE;
  const uint32_t bars = t_ring + S * t_stage;
  const uint32_t full0 = bars, empty0 = full0 + 8u * S, tail0 = empty0 + 8u * S;
  const uint32_t tfull0 = bars + 24u * kGroupedMaxStages, tempty0 = tfull0 + 16u;
  const uint32_t never_bar = tempty0 + 16u, holder = never_bar + 8u;
  volatile uint32_t* const holder_ptr = reinterpret_cast<volatile uint32_t*>(gbase + (holder - base));
  volatile uint32_t* const abort_ptr = holder_ptr + 1;
  int* const sums = reinterpret_cast<int*>(gbase + (holder + 16u - base));    // one per warp
  int* const offs = sums + 16;                   // clamped offsets, [groups + 1]
  int* const starts = offs + p.groups + 1;       // a group's first item, [groups + 1] (rows form)

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, kWeights ? CG : 1);
      mbar_init(empty0 + 8u * s, 1);
      mbar_init(tail0 + 8u * s, 1);
    }
    for (int a = 0; a < kAccStages; ++a) {
      mbar_init(tfull0 + 8u * a, 1);
      mbar_init(tempty0 + 8u * a, kGroupedEpiWarps * CG);
    }
    mbar_init(never_bar, 1);
    *abort_ptr = 0u;
    fence_barrier_init();
    if (p.has_operands) {
      prefetch_tensormap(&tmF);
      prefetch_tensormap(&tmT);
    }
  }
  if (warp == 1) {
    tmem_alloc<CG>(holder, kTmemCols);
    tmem_relinquish<CG>();
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = *holder_ptr;
  grid_dependency_wait();

  // The tables.  Offsets are clamped to the matrix and a negative size counts as
  // none, so that no offsets make an access out of range.
  const auto tiles_of = [&](int g, int rows) {
    if (p.skip_none && p.index) {
      const int e = __ldg(p.index + g);
      if (e < 0 || e >= p.sets) return 0;
    }
    return (rows + bn - 1) / bn;
  };
  for (int g = threadIdx.x; g <= p.groups; g += blockDim.x)
    offs[g] = min(max(__ldg(p.offsets + g), 0), p.rows);
  __syncthreads();
  int num_items = p.groups * p.tiles_f * p.tiles_c;
  if constexpr (!kWeights) {
    const int share = (p.groups + (int)blockDim.x - 1) / (int)blockDim.x;
    const int g0 = min((int)threadIdx.x * share, p.groups), g1 = min(g0 + share, p.groups);
    int mine = 0;
    for (int g = g0; g < g1; ++g) mine += tiles_of(g, max(0, offs[g + 1] - offs[g]));
    int upto = mine;                             // inclusive over the warp, then the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int at = upto - mine, total = 0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) {
      if (i < warp) at += sums[i];
      total += sums[i];
    }
    for (int g = g0; g < g1; ++g) {
      starts[g] = at * p.tiles_f;
      at += tiles_of(g, max(0, offs[g + 1] - offs[g]));
    }
    num_items = total * p.tiles_f;
    if (threadIdx.x == 0) starts[p.groups] = num_items;
    __syncthreads();
  }

  const Watch w{abort_ptr, p.status, p.timeout_ns};

  // An item: a feature tile of 128 CG features, and of its group either a tile of
  // tokens (the group's rows cut evenly, in whole units, into the fewest tiles of at
  // most bn) or a tile of output rows.
  struct Item {
    int g, e;                // group; set of weights, -1 for none
    int f0;                  // first feature
    int t0;                  // first token (rows form) or output row (weights form)
    int width, valid;        // MMA columns, and how many of them are the item's
    int m0, mn;              // weights form: the group's first row and number of rows
    int blocks;              // k-blocks
  };
  const int min_width = p.unit * CG;
  int cursor = 0;                                // the last item's group
  const auto item_at = [&](int it) {
    Item i;
    if constexpr (kWeights) {
      const int per = p.tiles_f * p.tiles_c;
      i.g = it / per;
      i.e = i.g;
      const int r = it - i.g * per;
      const int strip = r / (kGroupedStrip * p.tiles_f), rr = r - strip * kGroupedStrip * p.tiles_f;
      const int high = min(kGroupedStrip, p.tiles_c - strip * kGroupedStrip);
      i.f0 = rr / high * (128 * CG);
      i.t0 = (strip * kGroupedStrip + rr % high) * bn;
      i.valid = min(bn, p.cols - i.t0);
      i.width = (i.valid + min_width - 1) / min_width * min_width;
      i.m0 = offs[i.g];
      i.mn = max(0, offs[i.g + 1] - i.m0);
      i.blocks = (i.mn + BK - 1) / BK;
    } else {
      // starts[lo] <= it < starts[hi]; items come in increasing order
      int lo = cursor, hi = p.groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= it) lo = mid;
        else hi = mid;
      }
      cursor = lo;
      i.g = lo;
      i.e = p.index ? __ldg(p.index + lo) : lo;
      if (i.e < 0 || i.e >= p.sets) i.e = -1;
      const int rows = offs[lo + 1] - offs[lo];
      const int r = it - starts[lo], tiles = (rows + bn - 1) / bn;
      const int strip = r / (kGroupedStrip * p.tiles_f), rr = r - strip * kGroupedStrip * p.tiles_f;
      const int high = min(kGroupedStrip, tiles - strip * kGroupedStrip);
      const int tile = strip * kGroupedStrip + rr % high;
      i.f0 = rr / high * (128 * CG);
      const int each = ((rows + tiles - 1) / tiles + min_width - 1) / min_width * min_width;
      i.valid = max(0, min(each, rows - tile * each));
      i.width = max(min_width, (i.valid + min_width - 1) / min_width * min_width);
      i.t0 = offs[lo] + tile * each;
      i.m0 = i.mn = 0;
      i.blocks = i.e < 0 ? 0 : (p.k + BK - 1) / BK;
    }
    return i;
  };

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    const uint64_t pol = make_l2_policy(0);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int it = cluster_id; ok && it < num_items; it += num_clusters) {
      const Item i = item_at(it);
      const int f0 = i.f0 + (int)rank * 128;
      const int width = i.width / CG;                    // this CTA's columns
      const int t0 = i.t0 + (int)rank * width;
      for (int kb = 0; kb < i.blocks; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, wait_phase(empty0 + 8u * s, ph ^ 1u, w, kWaitProducer))) {
          ok = false;
          break;
        }
        const uint32_t sf = f_ring + s * F_STAGE, st = t_ring + s * t_stage;
        // (debug build, by every lane alike: the boxes inside this stage, coordinates whole 16
        // bytes and from 0 on)
        if (!dbg_check(in_range(sf, F_STAGE, f_ring, t_ring) && f0 >= 0, kChkLoadA, w) ||
            !dbg_check(in_range(st, (uint32_t)width * KA * 128u, t_ring, bars) && t0 >= 0 &&
                           i.m0 >= 0 && (!kWeights || t0 % 8 == 0),
                       kChkLoadB, w)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if constexpr (kWeights) {
            const int m = i.m0 + kb * BK;
            // both operands MN-major: boxes of 64 features or output rows x BK rows
            const uint32_t bytes = (uint32_t)(F_BOXES + width / ATOM_K) * MN_ATOM;
            const bool tail = kb == i.blocks - 1 && i.mn % UMMA_K != 0;
            if (tail) {
              // (completed on this CTA's own barrier: the zeroing warp goes on from there)
              const uint32_t bar = tail0 + 8u * s;
              mbar_arrive_expect_tx(bar, bytes);
              for (int j = 0; j < F_BOXES; ++j)
                tma_load_3d(sf + j * MN_ATOM, &tmF, bar, f0 + j * ATOM_K, m, 0, pol);
              for (int j = 0; j < width / ATOM_K; ++j)
                tma_load_3d(st + j * MN_ATOM, &tmT, bar, t0 + j * ATOM_K, m, 0, pol);
            } else {
              const uint32_t fb = full0 + 8u * s;
              const uint32_t bar = PAIR ? map_to_rank(fb, 0) : fb;
              if (rank == 0) mbar_arrive_expect_tx(fb, CG * bytes);
              else mbar_arrive_cluster(bar);
              for (int j = 0; j < F_BOXES; ++j)
                OperandLoad<CG, false>::load(sf + j * MN_ATOM, &tmF, bar, f0 + j * ATOM_K, m, 0, 0, pol);
              for (int j = 0; j < width / ATOM_K; ++j)
                OperandLoad<CG, false>::load(st + j * MN_ATOM, &tmT, bar, t0 + j * ATOM_K, m, 0, 0, pol);
            }
          } else {
            const int k0 = kb * BK;
            const int atoms = min(KA, (p.k - k0 + ATOM_K - 1) / ATOM_K);   // those with elements
            const uint32_t fb = full0 + 8u * s;
            const uint32_t bar = PAIR ? map_to_rank(fb, 0) : fb;
            if (rank == 0)
              mbar_arrive_expect_tx(fb, CG * ((p.f_mn ? F_STAGE : atoms * F_ATOM) +
                                              (uint32_t)(atoms * width) * 128u));
            if (p.f_mn) {
              for (int j = 0; j < F_BOXES; ++j)
                OperandLoad<CG, false>::load(sf + j * MN_ATOM, &tmF, bar, f0 + j * ATOM_K, k0, i.e, 0, pol);
            } else {
              for (int a = 0; a < atoms; ++a)
                OperandLoad<CG, false>::load(sf + a * F_ATOM, &tmF, bar, k0 + a * ATOM_K, f0, i.e, 0, pol);
            }
            for (int a = 0; a < atoms; ++a)
              for (int u = 0; u < width; u += p.unit)
                OperandLoad<CG, false>::load(st + a * t_atom + u * 128, &tmT, bar, k0 + a * ATOM_K,
                                             t0 + u, 0, 0, pol);
          }
        }
        __syncwarp();
        if (++s == S) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (rank == 0) {
      const bool f_mn = kWeights || p.f_mn;
      const uint64_t fd0 = f_mn ? smem_desc_sw128(f_ring, MN_ATOM, 1024)
                                : smem_desc_sw128(f_ring, 16, 1024);
      const uint64_t td0 = kWeights ? smem_desc_sw128(t_ring, MN_ATOM, 1024)
                                    : smem_desc_sw128(t_ring, 16, 1024);
      // 16-byte units from one K step to the next, and from one atom of steps to the next
      const uint32_t f_step = (f_mn ? UMMA_K * 128 : 32) / 16;
      const uint32_t t_step = (kWeights ? UMMA_K * 128 : 32) / 16;
      const uint32_t f_next = f_mn ? STEPS_PER_ATOM * f_step : F_ATOM / 16;
      const uint32_t t_next = kWeights ? STEPS_PER_ATOM * t_step : t_atom / 16;
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = !p.inject_stall ||
                __all_sync(0xFFFFFFFFu, wait_phase(never_bar, 0u, w, kWaitInjected));
      for (int it = cluster_id; ok && it < num_items; it += num_clusters) {
        const Item i = item_at(it);
        if (!__all_sync(0xFFFFFFFFu, wait_phase(tempty0 + 8u * acc, aph ^ 1u, w, kWaitMmaAcc)))
          break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + (uint32_t)acc * kAccStride;
        const uint32_t idesc = p.idesc | (uint32_t)(i.width >> 3) << 17;
        if (!dbg_check((uint32_t)i.width <= kAccStride, kChkMmaTmem, w)) break;
        for (int kb = 0; kb < i.blocks; ++kb) {
          ok = __all_sync(0xFFFFFFFFu, wait_phase(full0 + 8u * s, ph, w, kWaitMmaFull));
          if (!ok) break;
          tc_fence_after_sync();
          const uint64_t fd = fd0 + (uint32_t)(s * F_STAGE) / 16;
          const uint64_t td = td0 + (uint32_t)(s * t_stage) / 16;
          // the steps that hold elements (past them shared memory may hold anything)
          const int left = (kWeights ? i.mn : p.k) - kb * BK;
          const int steps = min(K_STEPS, (left + UMMA_K - 1) / UMMA_K);
          if constexpr (kDebug) {
            for (int k = 0; k < steps; ++k)
              ok = ok && dbg_check(desc_in_range(fd + (k / STEPS_PER_ATOM * f_next +
                                                       k % STEPS_PER_ATOM * f_step),
                                                 f_ring + s * F_STAGE, F_STAGE) &&
                                       desc_in_range(td + (k / STEPS_PER_ATOM * t_next +
                                                           k % STEPS_PER_ATOM * t_step),
                                                     t_ring + s * t_stage, t_stage),
                                   kChkMmaSmem, w);
            if (!ok) break;
          }
          if (elect_one()) {
            if (steps == K_STEPS) {
#pragma unroll
              for (int k = 0; k < K_STEPS; ++k)
                umma<CG, KIND>(d_tmem, fd + (k / STEPS_PER_ATOM * f_next + k % STEPS_PER_ATOM * f_step),
                               td + (k / STEPS_PER_ATOM * t_next + k % STEPS_PER_ATOM * t_step),
                               idesc, (kb | k) != 0 ? 1u : 0u);
            } else {
              for (int k = 0; k < steps; ++k)
                umma<CG, KIND>(d_tmem, fd + (k / STEPS_PER_ATOM * f_next + k % STEPS_PER_ATOM * f_step),
                               td + (k / STEPS_PER_ATOM * t_next + k % STEPS_PER_ATOM * t_step),
                               idesc, (kb | k) != 0 ? 1u : 0u);
            }
            umma_commit<CG, PAIR>(empty0 + 8u * s, 3);
          }
          __syncwarp();
          if (++s == S) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        if (elect_one()) umma_commit<CG, PAIR>(tfull0 + 8u * acc, 3);
        __syncwarp();
        if (++acc == kAccStages) { acc = 0; aph ^= 1u; }
      }
    }
  } else if (!kWeights || warp < 2 + kGroupedEpiWarps) {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;                      // TMEM lane quarter of this warp
    const int strm = (warp - 2) >> 2;
    int acc = 0, turn = 0;
    uint32_t aph = 0;
    const int r_es = p.r_dt == DT_F32 ? 4 : 2, z_es = p.z_dt == DT_F32 ? 4 : 2,
              d_es = p.d_dt == DT_F32 ? 4 : 2;
    const long long r_step = p.ldr * r_es, z_step = p.ldz * z_es, d_step = p.ldd * d_es;
    for (int it = cluster_id; it < num_items; it += num_clusters, turn ^= 1) {
      const Item i = item_at(it);
      const int f = i.f0 + (int)rank * 128 + q * 32 + lane;
      const bool mine = f < p.feats;
      // (debug build: what is stored lies inside d)
      if (!dbg_check(i.f0 >= 0 && i.t0 >= 0 && i.valid <= i.width &&
                         i.t0 + i.valid <= (kWeights ? p.cols : p.rows),
                     kChkEpiStore, w))
        break;
      const long long first = kWeights ? (long long)i.g * p.sd + (long long)i.t0 * p.ldd + f : 0;
      const long long row = i.t0;
      const uint8_t* const r_at = static_cast<const uint8_t*>(p.r) +
                                  (kWeights ? first * r_es : row * r_step + (long long)f * r_es);
      uint8_t* const z_at = static_cast<uint8_t*>(p.z) + (row * z_step + (long long)f * z_es);
      uint8_t* const d_at = static_cast<uint8_t*>(p.d) +
                            (kWeights ? first * d_es : row * d_step + (long long)f * d_es);
      const int count = mine ? i.valid : 0;
      float scale = p.alpha, bias = 0.f;
      if constexpr (!kWeights) {
        if (mine && i.e >= 0) {
          const long long at = (long long)i.e * p.feats + f;
          if (p.set_scale) scale *= __ldg(p.set_scale + i.e);
          if (p.col_scale) scale *= __ldg(p.col_scale + at);
          if (p.bias) bias = p.bias_dt == DT_F32 ? __ldg(static_cast<const float*>(p.bias) + at)
                             : p.bias_dt == DT_F16
                                 ? __half2float(__ushort_as_half(__ldg(static_cast<const uint16_t*>(p.bias) + at)))
                                 : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p.bias) + at) << 16);
        }
      }
      // Chunks of 16 columns, every other one this warp's; which warp of the two starts
      // alternates, so that items of one chunk are shared out.  A chunk's residual
      // and row factors (one a lane) are on their way before the accumulator is
      // waited for.
      uint32_t res[kGroupedChunk];
      float factor = 1.f;
      const auto fetch = [&](int c) {
        if (p.r) {
#pragma unroll
          for (int x = 0; x < kGroupedChunk; ++x)
            res[x] = c + x < count ? grouped_elem(r_at + (c + x) * r_step, p.r_dt) : 0u;
        }
        if constexpr (!kWeights) {
          if (p.row_scale && i.blocks > 0)
            factor = lane < kGroupedChunk && c + lane < i.valid
                         ? __ldg(p.row_scale + row + c + lane) : 1.f;
        }
      };
      const int c_first = (strm ^ turn) * kGroupedChunk;
      if (c_first < i.valid) fetch(c_first);
      if (!__all_sync(0xFFFFFFFFu, wait_phase(tfull0 + 8u * acc, aph, w, kWaitEpilogue))) break;
      tc_fence_after_sync();
      const auto release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) mbar_arrive(tempty0 + 8u * acc);
          else mbar_arrive_cluster(map_to_rank(tempty0 + 8u * acc, 0));
        }
      };
      if (c_first >= i.valid) release();
      const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * kAccStride;
#pragma unroll 1
      for (int c = c_first; c < i.valid; c += 2 * kGroupedChunk) {
        uint32_t a[kGroupedChunk];
        __syncwarp();
        tmem_load_16cols(tbase + c, a);
        tmem_wait_ld16(a);
        const bool last = c + 2 * kGroupedChunk >= i.valid;
        if (last) release();
        float v[kGroupedChunk];
#pragma unroll
        for (int x = 0; x < kGroupedChunk; ++x) v[x] = i.blocks ? __uint_as_float(a[x]) * scale : 0.f;
        if constexpr (!kWeights) {
          if (p.row_scale) {
#pragma unroll
            for (int x = 0; x < kGroupedChunk; ++x) v[x] *= __shfl_sync(0xFFFFFFFFu, factor, x);
          }
          if (p.bias) {
#pragma unroll
            for (int x = 0; x < kGroupedChunk; ++x) v[x] += bias;
          }
          if (p.z) grouped_store(z_at + c * z_step, z_step, p.z_dt, count - c, v);
          with_activation(p.act, [&](auto act) {
#pragma unroll
            for (int x = 0; x < kGroupedChunk; x += 2)
              activate2<decltype(act)::value>(v[x], v[x + 1]);
          });
        }
        if (p.r) {
          if (p.r_dt == DT_F32) {
#pragma unroll
            for (int x = 0; x < kGroupedChunk; ++x) v[x] += __uint_as_float(res[x]);
          } else if (p.r_dt == DT_F16) {
#pragma unroll
            for (int x = 0; x < kGroupedChunk; ++x)
              v[x] += __half2float(__ushort_as_half((uint16_t)res[x]));
          } else {
#pragma unroll
            for (int x = 0; x < kGroupedChunk; ++x) v[x] += __uint_as_float(res[x] << 16);
          }
        }
        if (!last) fetch(c + 2 * kGroupedChunk);
        grouped_store(d_at + c * d_step, d_step, p.d_dt, count - c, v);
      }
      if (++acc == kAccStages) { acc = 0; aph ^= 1u; }
    }
  } else {
    // ---------------------------------------------------------- zeroing (weights form)
    int s = 0;
    uint32_t phases = 0;                         // a bit per stage: its tail barrier's phase
    for (int it = cluster_id; it < num_items; it += num_clusters) {
      const Item i = item_at(it);
      if (i.blocks > 0 && i.mn % UMMA_K != 0) {
        const int at = (s + i.blocks - 1) % S;
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(tail0 + 8u * at, phases >> at & 1u, w,
                                                      kWaitProducer)))
          break;
        phases ^= 1u << at;
        // rows [from, to) of every 128-byte wide atom column
        const int from = i.mn - (i.blocks - 1) * BK, to = (from + UMMA_K - 1) / UMMA_K * UMMA_K;
        uint8_t* const sf = gbase + (f_ring + at * F_STAGE - base);
        uint8_t* const st = gbase + (t_ring + at * t_stage - base);
        const int boxes = i.width / CG / ATOM_K;
        for (int j = 0; j < F_BOXES + boxes; ++j) {
          uint8_t* const box = j < F_BOXES ? sf + j * MN_ATOM : st + (j - F_BOXES) * MN_ATOM;
          for (int b = from * 128 + lane * 16; b < to * 128; b += 512)
            *reinterpret_cast<uint4*>(box + b) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_all();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) mbar_arrive(full0 + 8u * at);
          else mbar_arrive_cluster(map_to_rank(full0 + 8u * at, 0));
        }
      }
      s = (s + i.blocks) % S;
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (*abort_ptr) {
    // A wait gave up: let copies and MMAs already issued drain first.
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  __syncwarp();
  if constexpr (PAIR) cluster_sync_all();        // the other CTA may still use this one's memory
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<CG>(tmem_base, kTmemCols);
  }
}

}  // namespace gb300
