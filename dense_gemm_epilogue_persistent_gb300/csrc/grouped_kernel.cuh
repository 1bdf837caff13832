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
// columns.  A tile's width then follows its group in steps of 16 columns (32 of single CTAs'
// tiles wider than 64, 64 of pairs' and in the weights form of each CTA's), so
// that a ragged group costs little more than its own rows; an accumulator column is
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
// stage's copies report to a barrier of the CTA, the other CTA's zeroing warp to the
// leader's, which then completes the stage.  (A remote arrival for every stage instead, to
// have the stages count both CTAs, cost a quarter: 8192^3 bf16 880 us, 648 so.)
//
// Both gradients of a layer run as one launch: the items of da (rows), then those of db
// (weights), dealt to the CTAs in one sequence, so that a launch's start and end and the
// first product's last, partial round are paid once.
//
// Block: warp 0 TMA producer, warp 1 tensor memory and MMA issue, then the epilogue's (two warps
// per lane quarter, three where its code is lean, taking 32-column chunks in turn) and,
// with a weights form, the zeroing.  Persistent grid of CTAs or CTA pairs, one CTA an
// SM, two accumulator stages.  Bound by the operands' way out of L2 for large groups (a stage of a
// 256 x 256 pair tile takes 1230 cycles for 64 KB, 1024 of MMA), by the weights' DRAM traffic for small
// ones.  The waits are bounded as in gemm_kernel.cuh.
#pragma once

#include "activations.cuh"
#include "gemm_kernel.cuh"

namespace gb300 {

// n / d for 0 <= n < 2^31 by a multiplication: with 2^s >= d > 2^(s-1) and m = ceil(2^(31+s) / d),
// floor(n m / 2^(31+s)) is exact, since m d - 2^(31+s) < d <= 2^s.
struct FastDiv {
  uint32_t mul, shift;
  int d;
};
inline FastDiv fast_div(int d) {
  uint32_t s = 0;
  while ((1ull << s) < (unsigned long long)d) ++s;
  return {(uint32_t)(((1ull << (31 + s)) + (unsigned long long)d - 1) / (unsigned long long)d), 31 + s, d};
}
__device__ __forceinline__ int fast_quot(int n, const FastDiv& f) {
  return (int)(((unsigned long long)(uint32_t)n * f.mul) >> f.shift);
}

struct GroupedParams {
  int rows;                  // of the token matrix: groups are clamped to them
  int feats;                 // output features (MMA rows)
  int cols;                  // weights form: output rows of a group (MMA columns)
  int k;                     // rows form: inner size
  int groups, sets;          // groups of rows, sets of weights
  int bn;                    // widest tile
  int unit;                  // columns of one box of the token operand
  int f_rows;                // features of a stage: 128, or of a single narrow tile of K-major weights its
                             // own (the MMA reads 128 rows of shared memory all the same; what it
                             // makes of the others is not stored)
  int tiles_f, tiles_c;      // feature tiles; weights form: column tiles
  FastDiv by_bn, by_strip, by_group;   // by bn, a whole strip's items, a group's (weights form)
  int stages;
  int alternate;             // odd waves of items walk the k-blocks from the last one down (8192^3 bf16
                             // 659 us, 675 without)
  int strip;                 // token (or column) tiles walked together
  int set_step;              // 0: all sets are one matrix
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

// Both forms in one launch: the rows form's, whose tile, ring and groups are common, and the
// weights form's with its tensor maps.
struct GroupedBothParams : GroupedParams {
  GroupedParams weights;
  CUtensorMap f2, t2;
};
enum : int { kGroupedRows = 0, kGroupedWeights = 1, kGroupedBoth = 2 };
template <int FORM> struct GroupedParamsOf { using type = GroupedParams; };
template <> struct GroupedParamsOf<kGroupedBoth> { using type = GroupedBothParams; };
__device__ __forceinline__ const GroupedParams& weights_of(const GroupedParams& p) { return p; }
__device__ __forceinline__ const GroupedParams& weights_of(const GroupedBothParams& p) { return p.weights; }
__device__ __forceinline__ const CUtensorMap* second_map(const GroupedParams&, const CUtensorMap& map, int) {
  return &map;
}
__device__ __forceinline__ const CUtensorMap* second_map(const GroupedBothParams& p, const CUtensorMap&, int i) {
  return i ? &p.t2 : &p.f2;
}

constexpr int kGroupedKA = 2;                  // 128-byte K atoms a ring stage
constexpr int kGroupedMBox = 128;              // rows of one box of the weights form, a stage's (boxes of 64: 16
                                               // groups 245 -> 258 us)
constexpr int kGroupedChunk = 32;              // columns of an epilogue chunk
constexpr int kGroupedMaxStrip = 16;
constexpr int kGroupedMaxGroups = 4096;        // what the tables in shared memory hold
constexpr int kGroupedMaxStages = 10;

// Epilogue warps per tensor-memory lane quarter: three where the lean epilogue's registers allow it
// (64 groups' weight gradients of 128 rows, 4096 x 4096 bf16: 457 us, 549 with two).
__host__ __device__ constexpr int grouped_streams(int lean) { return lean >= 0 ? 3 : 2; }
constexpr int grouped_threads(int form, int lean) {
  return 64 + 128 * grouped_streams(lean) + (form == kGroupedRows ? 0 : 32);
}

// Bytes of a ring stage and of what follows the ring: barriers (full, empty, tail, peer; two
// accumulators' full and empty; one that nothing arrives at), tensor-memory
// address and abort flag, warps' sums, reciprocals, the two tables.
constexpr int grouped_stage_bytes(int cta_group, int bn, int f_rows) {
  return kGroupedKA * (f_rows + bn / cta_group) * 128;
}
constexpr int grouped_bar_bytes() { return 8 * (4 * kGroupedMaxStages + 5) + 16 + 128 + 80; }
constexpr int grouped_smem(int cta_group, int bn, int f_rows, int stages, int groups) {
  return 1024 + stages * grouped_stage_bytes(cta_group, bn, f_rows) + grouped_bar_bytes() +
         8 * (groups + 1);
}

// Where a lane's values of the columns (tokens) of a matrix lie.  With 16 bits two neighbouring
// lanes exchange halves of two columns x, x + 1, so that each moves two neighbouring
// features, 4 bytes, of one of them: even lanes of x, odd lanes of x + 1.  (A quarter fewer
// instructions than 2 bytes of each.)  That is the way of whole chunks (`pairs`); where columns or
// the last of an odd number of features are missing every lane moves its own elements.
__host__ __device__ constexpr int elem_size(int dt) { return dt == DT_F32 ? 4 : 2; }
struct EpiMatrix {
  uint8_t* own;              // this lane's element of column 0
  uint8_t* pair;             // the two elements that it moves of columns 0, 1
  long long step;            // bytes from one column to the next
  int dt;
};
__device__ __forceinline__ uint32_t swap_halves(uint32_t w, uint32_t odd) {
  return __byte_perm(w, __shfl_xor_sync(0xFFFFFFFFu, w, 1), odd ? 0x3276 : 0x5410);
}

// 16 columns from c on, of which `left` are the item's, for lanes that have a feature (mine).
// (One way through each of the two forms, its stores predicated by column: code that is run
// once a chunk is fetched from memory as often as it is run.)
__device__ __forceinline__ void epi_store(const EpiMatrix& m, int c, int left, bool pairs, bool mine,
                                          uint32_t odd, const float (&v)[16]) {
  if (m.dt == DT_F32) {
    uint8_t* p = m.own + c * m.step;
#pragma unroll
    for (int x = 0; x < 16; ++x, p += m.step)
      if (mine && x < left) *reinterpret_cast<float*>(p) = v[x];
    return;
  }
  uint32_t w[8];
  if (m.dt == DT_F16) {
#pragma unroll
    for (int x = 0; x < 8; ++x) w[x] = pack_f16x2(v[2 * x], v[2 * x + 1]);
  } else {
#pragma unroll
    for (int x = 0; x < 8; ++x) w[x] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
  }
  if (pairs) {
#pragma unroll
    for (int x = 0; x < 8; ++x) w[x] = swap_halves(w[x], odd);
    const int mine_left = mine ? left - (int)odd : 0;
    uint8_t* p = m.pair + c * m.step;
#pragma unroll
    for (int x = 0; x < 8; ++x, p += 2 * m.step)
      if (2 * x < mine_left) *reinterpret_cast<uint32_t*>(p) = w[x];
  } else {
    uint8_t* p = m.own + c * m.step;
#pragma unroll
    for (int x = 0; x < 16; ++x, p += m.step)
      if (mine && x < left) *reinterpret_cast<uint16_t*>(p) = (uint16_t)(w[x / 2] >> (16 * (x & 1)));
  }
}

// The words of such 16 columns, as they lie in memory: 16 of 32 bits, or 8 of two columns of 16.
template <int FROM>
__device__ __forceinline__ void epi_load(const EpiMatrix& m, int c, int left, bool pairs, bool mine,
                                         uint32_t odd, uint32_t (&r)[32]) {
  if (m.dt == DT_F32) {
    const uint8_t* p = m.own + c * m.step;
#pragma unroll
    for (int x = 0; x < 16; ++x, p += m.step)
      r[(FROM + x) & 31] = mine && x < left ? *reinterpret_cast<const uint32_t*>(p) : 0u;
  } else if (pairs) {
    const int mine_left = mine ? left - (int)odd : 0;
    const uint8_t* p = m.pair + c * m.step;
#pragma unroll
    for (int x = 0; x < 8; ++x, p += 2 * m.step)
      r[(FROM + x) & 31] = 2 * x < mine_left ? *reinterpret_cast<const uint32_t*>(p) : 0u;
  } else {
    const uint8_t* p = m.own + c * m.step;
#pragma unroll
    for (int x = 0; x < 8; ++x, p += 2 * m.step) {
      const uint32_t lo = mine && 2 * x < left ? *reinterpret_cast<const uint16_t*>(p) : 0u;
      const uint32_t hi =
          mine && 2 * x + 1 < left ? *reinterpret_cast<const uint16_t*>(p + m.step) : 0u;
      r[(FROM + x) & 31] = lo | hi << 16;
    }
  }
}
template <int FROM>
__device__ __forceinline__ void epi_add(const EpiMatrix& m, bool pairs, uint32_t odd,
                                        const uint32_t (&r)[32], float (&v)[16]) {
  if (m.dt == DT_F32) {
#pragma unroll
    for (int x = 0; x < 16; ++x) v[x] += __uint_as_float(r[(FROM + x) & 31]);
    return;
  }
  uint32_t w[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) w[x] = r[(FROM + x) & 31];
  if (pairs) {
#pragma unroll
    for (int x = 0; x < 8; ++x) w[x] = swap_halves(w[x], odd);
  }
  if (m.dt == DT_F16) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float2 f = unpack_f16x2(w[x]);
      v[2 * x] += f.x;
      v[2 * x + 1] += f.y;
    }
  } else {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float2 f = unpack_bf16x2(w[x]);
      v[2 * x] += f.x;
      v[2 * x + 1] += f.y;
    }
  }
}

// LEAN < 0: the whole epilogue, every type.  Else nothing but alpha, a set's scale and a residual
// follow the product, d and the residual are of type LEAN, and with a 16-bit residual the number of
// features is even.
template <int CG, int AB_BYTES, int FORM, int LEAN>
__global__ void __launch_bounds__(grouped_threads(FORM, LEAN), 1)
grouped_kernel(const __grid_constant__ CUtensorMap tmF, const __grid_constant__ CUtensorMap tmT,
               const __grid_constant__ CUtensorMap tmWhole,
               const __grid_constant__ typename GroupedParamsOf<FORM>::type p) {
  constexpr bool kRows = FORM != kGroupedWeights, kWeights = FORM != kGroupedRows;
  constexpr bool kFull = FORM == kGroupedRows && LEAN < 0;
  constexpr int KIND = (AB_BYTES == 1) ? 1 : (AB_BYTES == 4 ? 2 : 0);
  constexpr int KA = kGroupedKA;
  constexpr int ATOM_K = 128 / AB_BYTES;         // K of a 128-byte atom; features of an MN-major one
  constexpr int BK = ATOM_K * KA;                // inner size of a stage
  constexpr int UMMA_K = 32 / AB_BYTES;
  constexpr int K_STEPS = BK / UMMA_K;
  constexpr int STEPS_PER_ATOM = ATOM_K / UMMA_K;
  constexpr uint32_t MN_ATOM = BK * 128;         // bytes of an MN-major atom column
  constexpr int F_BOXES = 128 / ATOM_K;          // MN-major boxes of the 128 features
  constexpr bool PAIR = CG == 2;
  constexpr int kStreams = grouped_streams(LEAN), kEpiWarps = 4 * kStreams;
  static_assert(!kWeights || AB_BYTES == 2, "weight gradients are of 16-bit operands");
  static_assert(FORM != kGroupedBoth || LEAN >= 0, "both forms: the lean epilogue");
  static_assert(BK == kGroupedMBox || !kWeights, "a stage's rows in one box");

  grid_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // the same in both CTAs of a pair
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int cluster_id = blockIdx.x / CG, num_clusters = gridDim.x / CG;
  const GroupedParams& pw = weights_of(p);       // the weights form's
  const int S = p.stages, bn = p.bn;
  const uint32_t t_atom = (uint32_t)(bn / CG) * 128u;    // K-major atom of the CTA's tokens
  const uint32_t t_stage = t_atom * KA;
  const uint32_t f_atom = (uint32_t)p.f_rows * 128u;     // ... of its features (MN-major: 128 of them)
  const uint32_t f_stage = f_atom * KA;
  const uint32_t f_ring = base, t_ring = f_ring + S * f_stage;
  const uint32_t bars = t_ring + S * t_stage;
  const uint32_t full0 = bars, empty0 = full0 + 8u * S, tail0 = empty0 + 8u * S;
  const uint32_t peer0 = tail0 + 8u * S;         // the other CTA's half of a last block is zeroed
  const uint32_t tfull0 = bars + 32u * kGroupedMaxStages, tempty0 = tfull0 + 16u;
  const uint32_t never_bar = tempty0 + 16u, holder = never_bar + 8u;
  volatile uint32_t* const holder_ptr = reinterpret_cast<volatile uint32_t*>(gbase + (holder - base));
  volatile uint32_t* const abort_ptr = holder_ptr + 1;
  long long* const sums = reinterpret_cast<long long*>(gbase + (holder + 16u - base));    // one per warp
  uint32_t* const magic = reinterpret_cast<uint32_t*>(sums + 16);     // ceil(2^32 / n), [17]
  int* const offs = reinterpret_cast<int*>(magic) + 20;        // clamped offsets, [groups + 1]
  int* const starts = offs + p.groups + 1;       // a group's first item, [groups + 1] (rows form)

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
      mbar_init(tail0 + 8u * s, 1);
      mbar_init(peer0 + 8u * s, 1);
    }
    for (int a = 0; a < kAccStages; ++a) {
      mbar_init(tfull0 + 8u * a, 1);
      mbar_init(tempty0 + 8u * a, kEpiWarps * CG);
    }
    mbar_init(never_bar, 1);
    *abort_ptr = 0u;
    fence_barrier_init();
    if (p.has_operands) {
      prefetch_tensormap(&tmF);
      prefetch_tensormap(&tmT);
      if constexpr (kRows) prefetch_tensormap(&tmWhole);
    }
    if constexpr (FORM == kGroupedBoth) {
      prefetch_tensormap(&p.f2);
      prefetch_tensormap(&p.t2);
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
    return fast_quot(rows + bn - 1, p.by_bn);
  };
  // (rr / high by __umulhi(rr, magic[high]): exact below 2^28, which holds 16 x the feature tiles)
  if (threadIdx.x >= 2 && threadIdx.x <= kGroupedMaxStrip)
    magic[threadIdx.x] = 0xFFFFFFFFu / threadIdx.x + 1u;
  for (int g = threadIdx.x; g <= p.groups; g += blockDim.x)
    offs[g] = min(max(__ldg(p.offsets + g), 0), p.rows);
  __syncthreads();
  int rows_items = 0;
  if constexpr (kRows) {
    const int share = (p.groups + (int)blockDim.x - 1) / (int)blockDim.x;
    const int g0 = min((int)threadIdx.x * share, p.groups), g1 = min(g0 + share, p.groups);
    // (64 bits: groups that lie on one another may together hold any number of tiles; those past
    // 2^30 items are left out)
    const auto items_to = [&](long long tiles) { return (int)min(tiles * p.tiles_f, 1ll << 30); };
    long long mine = 0;
    for (int g = g0; g < g1; ++g) mine += tiles_of(g, max(0, offs[g + 1] - offs[g]));
    long long upto = mine;                       // inclusive over the warp, then the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long at = upto - mine, total = 0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) {
      if (i < warp) at += sums[i];
      total += sums[i];
    }
    for (int g = g0; g < g1; ++g) {
      starts[g] = items_to(at);
      at += tiles_of(g, max(0, offs[g + 1] - offs[g]));
    }
    rows_items = items_to(total);
    if (threadIdx.x == 0) starts[p.groups] = rows_items;
    __syncthreads();
  }
  const int weights_items = kWeights ? pw.groups * pw.tiles_f * pw.tiles_c : 0;
  const int num_items = rows_items + weights_items;

  // The CTA's (pair's) sequence of items.  They are dealt in turn; with both forms, the CTAs that got
  // one of the rows form's less have first of the others as many as take about as long (a
  // stage takes 1230 cycles, an epilogue that no main loop hides 3000).
  int lead = 0, lead_from = 0;                   // so many items ahead, to the CTAs from lead_from on
  if constexpr (FORM == kGroupedBoth) {
    lead_from = rows_items % num_clusters;
    if (lead_from > 0) {
      const int behind = num_clusters - lead_from;
      // (cycles in 64 bits: 224 million features are 2^31 of them)
      const int mean = (offs[p.groups] - offs[0]) / p.groups;
      const long long one = max(1230ll * ((mean + BK - 1) / BK), 3000ll);
      const long long rounds = (1230ll * ((p.k + BK - 1) / BK) + 3000) / one;
      lead = (int)min(rounds, (long long)(weights_items / behind)) * behind;
    }
  }
  const auto second_item = [&]() {
    return lead > 0 && cluster_id >= lead_from ? rows_items + cluster_id - lead_from
                                               : rows_items + lead + cluster_id;
  };
  const auto next_item = [&](int it) {
    if constexpr (FORM == kGroupedBoth) {
      if (it < rows_items) return it + num_clusters < rows_items ? it + num_clusters : second_item();
      if (it < rows_items + lead) {
        const int next = it + num_clusters - lead_from;
        return next < rows_items + lead ? next : rows_items + lead + cluster_id;
      }
    }
    return it + num_clusters;
  };
  const int first_item = FORM == kGroupedBoth && cluster_id >= rows_items ? second_item() : cluster_id;

  const Watch w{abort_ptr, p.status, p.timeout_ns};

  // An item: a feature tile of 128 CG features, and of its group either a tile of up to bn
  // tokens (all but a group's last one bn wide) or a tile of output rows.  Items of a group
  // go through its strips of `strip` token (or column) tiles, tile by tile, then feature by
  // feature, so that CTAs at work together share operands in L2.
  struct Item {
    bool wt;                 // of the weights form
    int g, e;                // group; set of weights, -1 for none
    int f0;                  // first feature
    int t0;                  // first token (rows form) or output row (weights form)
    int width, valid;        // MMA columns, and how many of them are the item's
    int m0, mn;              // weights form: the group's first row and number of rows
    int blocks;              // k-blocks
    bool down;               // walked from the last one
  };
  const int k_blocks = (p.k + BK - 1) / BK;
  int cursor = 0, wave = 0;                      // the last item's group; items so far
  const auto item_at = [&](int it) {
    Item i;
    i.wt = FORM == kGroupedBoth ? it >= rows_items : kWeights;
    i.down = p.alternate && (wave++ & 1);
    const GroupedParams& q = i.wt ? pw : p;
    int r, tiles;
    if (kWeights && i.wt) {
      i.g = fast_quot(it - rows_items, q.by_group);
      r = it - rows_items - i.g * q.by_group.d;
      tiles = q.tiles_c;
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
      r = it - starts[lo];
      tiles = fast_quot(offs[lo + 1] - offs[lo] + bn - 1, p.by_bn);
    }
    const int strip = fast_quot(r, q.by_strip), rr = r - strip * q.by_strip.d;
    const int high = min(q.strip, tiles - strip * q.strip);
    const int ft = high == 1 ? rr : (int)__umulhi((uint32_t)rr, magic[high]);
    const int tile = strip * q.strip + rr - ft * high;
    i.f0 = ft * (128 * CG);
    if (kWeights && i.wt) {
      i.e = i.g;
      i.t0 = tile * bn;
      i.valid = min(bn, q.cols - i.t0);
      i.m0 = offs[i.g];
      i.mn = max(0, offs[i.g + 1] - i.m0);
      i.blocks = (i.mn + BK - 1) / BK;
    } else {
      i.e = p.index ? __ldg(p.index + i.g) : i.g;
      if (i.e < 0 || i.e >= p.sets) i.e = -1;
      i.t0 = offs[i.g] + tile * bn;
      i.valid = min(bn, offs[i.g + 1] - i.t0);
      i.m0 = i.mn = 0;
      i.blocks = i.e < 0 ? 0 : k_blocks;
    }
    const int min_width = q.unit * CG;           // (a power of two)
    i.width = (i.valid + min_width - 1) & -min_width;
    return i;
  };

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    const uint64_t pol = make_l2_policy(0);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int it = first_item; ok && it < num_items; it = next_item(it)) {
      const Item i = item_at(it);
      const int f0 = i.f0 + (int)rank * 128;
      const int width = i.width / CG;                    // this CTA's columns
      const int t0 = i.t0 + (int)rank * width;
      for (int n = 0; n < i.blocks; ++n) {
        const int kb = i.down ? i.blocks - 1 - n : n;
        if (!__all_sync(0xFFFFFFFFu, wait_phase(empty0 + 8u * s, ph ^ 1u, w, kWaitProducer))) {
          ok = false;
          break;
        }
        const uint32_t sf = f_ring + s * f_stage, st = t_ring + s * t_stage;
        // (debug build, by every lane alike: the boxes inside this stage, coordinates whole 16
        // bytes and from 0 on)
        if (!dbg_check(in_range(sf, f_stage, f_ring, t_ring) && f0 >= 0, kChkLoadA, w) ||
            !dbg_check(in_range(st, (uint32_t)width * KA * 128u, t_ring, bars) && t0 >= 0 &&
                           i.m0 >= 0 && (!i.wt || t0 % 8 == 0),
                       kChkLoadB, w)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (kWeights && i.wt) {
            // both operands MN-major: boxes of 64 features or output rows x the stage's rows
            const CUtensorMap* const map_f = second_map(p, tmF, 0);
            const CUtensorMap* const map_t = second_map(p, tmT, 1);
            const int m = i.m0 + kb * BK, left = i.mn - kb * BK;
            const uint32_t bytes = (uint32_t)(F_BOXES + width / ATOM_K) * MN_ATOM;
            const bool tail = left <= BK && i.mn % UMMA_K != 0;
            // (a last block that needs zeros is completed on this CTA's own barrier: the zeroing
            // warp goes on from there)
            const uint32_t fb = full0 + 8u * s;
            const uint32_t bar = tail ? tail0 + 8u * s : PAIR ? map_to_rank(fb, 0) : fb;
            if (tail) mbar_arrive_expect_tx(bar, bytes);
            else if (rank == 0) mbar_arrive_expect_tx(fb, CG * bytes);
            for (int j = 0; j < F_BOXES; ++j) {
              if (tail) tma_load_3d(sf + j * MN_ATOM, map_f, bar, f0 + j * ATOM_K, m, 0, pol);
              else OperandLoad<CG, false>::load(sf + j * MN_ATOM, map_f, bar, f0 + j * ATOM_K, m, 0, 0, pol);
            }
            for (int j = 0; j < width / ATOM_K; ++j) {
              if (tail) tma_load_3d(st + j * MN_ATOM, map_t, bar, t0 + j * ATOM_K, m, 0, pol);
              else OperandLoad<CG, false>::load(st + j * MN_ATOM, map_t, bar, t0 + j * ATOM_K, m, 0, 0, pol);
            }
          } else if (kRows) {
            const int k0 = kb * BK, set = i.e * p.set_step;
            const int atoms = min(KA, (p.k - k0 + ATOM_K - 1) / ATOM_K);   // those with elements
            const uint32_t fb = full0 + 8u * s;
            const uint32_t bar = PAIR ? map_to_rank(fb, 0) : fb;
            if (rank == 0)
              mbar_arrive_expect_tx(fb, CG * ((p.f_mn ? f_stage : (uint32_t)atoms * f_atom) +
                                              (uint32_t)(atoms * width) * 128u));
            if (p.f_mn) {
              for (int j = 0; j < F_BOXES; ++j)
                OperandLoad<CG, false>::load(sf + j * MN_ATOM, &tmF, bar, f0 + j * ATOM_K, k0, set, 0, pol);
            } else {
              for (int a = 0; a < atoms; ++a)
                OperandLoad<CG, false>::load(sf + a * f_atom, &tmF, bar, k0 + a * ATOM_K, f0, set, 0, pol);
            }
            // a whole tile's tokens in one box an atom, else in units (adapters' first product, 8191
            // rows of 4096 by 7 x 64 bf16: 21.5 us, 22.5 in units alone; 8192^3 659, 673)
            if (i.width == bn) {
              for (int a = 0; a < atoms; ++a)
                OperandLoad<CG, false>::load(st + a * t_atom, &tmWhole, bar, k0 + a * ATOM_K, t0, 0, 0, pol);
            } else {
              for (int a = 0; a < atoms; ++a)
                for (int u = 0; u < width; u += p.unit)
                  OperandLoad<CG, false>::load(st + a * t_atom + u * 128, &tmT, bar, k0 + a * ATOM_K,
                                               t0 + u, 0, 0, pol);
            }
          }
        }
        __syncwarp();
        if (++s == S) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (rank == 0) {
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = !p.inject_stall ||
                __all_sync(0xFFFFFFFFu, wait_phase(never_bar, 0u, w, kWaitInjected));
      for (int it = first_item; ok && it < num_items; it = next_item(it)) {
        const Item i = item_at(it);
        const bool wt = kWeights && i.wt, f_mn = wt || p.f_mn;
        const uint64_t fd0 = f_mn ? smem_desc_sw128(f_ring, MN_ATOM, 1024)
                                  : smem_desc_sw128(f_ring, 16, 1024);
        const uint64_t td0 = wt ? smem_desc_sw128(t_ring, MN_ATOM, 1024)
                                : smem_desc_sw128(t_ring, 16, 1024);
        // 16-byte units from one K step to the next, and from one atom of steps to the next
        const uint32_t f_step = (f_mn ? UMMA_K * 128 : 32) / 16;
        const uint32_t t_step = (wt ? UMMA_K * 128 : 32) / 16;
        const uint32_t f_next = f_mn ? STEPS_PER_ATOM * f_step : f_atom / 16;
        const uint32_t t_next = wt ? STEPS_PER_ATOM * t_step : t_atom / 16;
        if (!__all_sync(0xFFFFFFFFu, wait_phase(tempty0 + 8u * acc, aph ^ 1u, w, kWaitMmaAcc)))
          break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + (uint32_t)acc * kAccStride;
        const uint32_t idesc = (wt ? pw.idesc : p.idesc) | (uint32_t)(i.width >> 3) << 17;
        if (!dbg_check((uint32_t)i.width <= kAccStride, kChkMmaTmem, w)) break;
        for (int n = 0; n < i.blocks; ++n) {
          const int kb = i.down ? i.blocks - 1 - n : n;
          ok = __all_sync(0xFFFFFFFFu, wait_phase(full0 + 8u * s, ph, w, kWaitMmaFull));
          if (!ok) break;
          tc_fence_after_sync();
          const uint64_t fd = fd0 + (uint32_t)(s * f_stage) / 16;
          const uint64_t td = td0 + (uint32_t)(s * t_stage) / 16;
          // the steps that hold elements (past them shared memory may hold anything)
          const int left = (wt ? i.mn : p.k) - kb * BK;
          const int steps = min(K_STEPS, (left + UMMA_K - 1) / UMMA_K);
          if constexpr (kDebug) {
            for (int k = 0; k < steps; ++k)
              ok = ok && dbg_check(desc_in_range(fd + (k / STEPS_PER_ATOM * f_next +
                                                       k % STEPS_PER_ATOM * f_step),
                                                 f_ring + s * f_stage, f_stage) &&
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
                               idesc, (n | k) != 0 ? 1u : 0u);
            } else {
              for (int k = 0; k < steps; ++k)
                umma<CG, KIND>(d_tmem, fd + (k / STEPS_PER_ATOM * f_next + k % STEPS_PER_ATOM * f_step),
                               td + (k / STEPS_PER_ATOM * t_next + k % STEPS_PER_ATOM * t_step),
                               idesc, (n | k) != 0 ? 1u : 0u);
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
  } else if (warp < 2 + kEpiWarps) {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;                      // TMEM lane quarter of this warp
    const int strm = (warp - 2) >> 2;
    const uint32_t odd = lane & 1;
    int acc = 0, turn = 0;                       // turn: the stream that takes the item's first chunk
    uint32_t aph = 0;
    constexpr int kNext = kStreams * kGroupedChunk;      // from one of this warp's chunks to the next
    const auto first_chunk = [&](int t) {
      return (strm >= t ? strm - t : strm - t + kStreams) * kGroupedChunk;
    };
    const auto next_turn = [&](int t) { return t + 1 == kStreams ? 0 : t + 1; };
    // The accumulator's columns have been read.  (The arrival hands over nothing but these, whose
    // loads have completed; the pair's leader may be the other CTA.)
    const auto release = [&]() {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 1) mbar_arrive(tempty0 + 8u * acc);
        else mbar_arrive_cluster_relaxed(map_to_rank(tempty0 + 8u * acc, 0));
      }
    };
    if constexpr (LEAN >= 0) {
      constexpr int ES = elem_size(LEAN), W = ES == 4 ? 16 : 8;    // words of 16 columns
      constexpr int PER = 16 / W;                // columns from one of a lane's words to the next
      const uint32_t second = PER == 2 ? odd : 0u;
      // An item and this lane's place in it.
      struct At {
        Item i;
        bool mine, has_r;
        bool odd_feats;        // 16 bits: an odd number of features, moved one by one
        float scale;
        const uint8_t* r;
        uint8_t* d;
        long long r_step, d_step;
      };
      const auto at_item = [&](int it) {
        At t;
        t.i = item_at(it);
        const int f = t.i.f0 + (int)rank * 128 + q * 32 + lane;
        const GroupedParams& o = t.i.wt ? pw : p;
        const long long group = t.i.wt ? (long long)t.i.g * o.sd : 0ll;
        t.odd_feats = PER == 2 && (o.feats & 1);
        const bool pairs = PER == 2 && !t.odd_feats;
        const long long row = t.i.t0 + (pairs ? second : 0u), col = pairs ? f & ~1 : f;
        t.has_r = o.r != nullptr;
        t.r_step = o.ldr * ES;
        t.d_step = o.ldd * ES;
        t.r = static_cast<const uint8_t*>(o.r) + (group + row * o.ldr + col) * ES;
        t.d = static_cast<uint8_t*>(o.d) + (group + row * o.ldd + col) * ES;
        t.mine = f < o.feats;
        t.scale = t.i.blocks ? o.alpha : 0.f;
        if constexpr (kRows) {
          if (!t.i.wt && p.set_scale && t.i.blocks) t.scale *= __ldg(p.set_scale + t.i.e);
        }
        return t;
      };
      // The residual's words of 16 columns, `left` of them there, from `at` on.
      uint32_t res[2 * W];
      const auto fetch = [&](auto from, const uint8_t* at, long long step, int left) {
        constexpr int FROM = decltype(from)::value;
#pragma unroll
        for (int x = 0; x < W; ++x, at += PER * step) {
          res[FROM + x] = 0u;
          if (PER * x + (int)second < left) res[FROM + x] = *reinterpret_cast<const uint32_t*>(at);
        }
      };
      At t{};
      const auto fetch_first = [&](const At& a, int c) {
        if (!a.has_r) return;
        fetch(IntC<0>{}, a.r + c * a.r_step, a.r_step, a.mine ? a.i.valid - c : 0);
        fetch(IntC<W>{}, a.r + (c + 16) * a.r_step, a.r_step, a.mine ? a.i.valid - c - 16 : 0);
      };
      if (first_item < num_items) {
        t = at_item(first_item);
        fetch_first(t, first_chunk(turn));
      }
      for (int it = first_item, it_next; it < num_items; it = it_next, turn = next_turn(turn)) {
        // The next item, its residual on its way into L2 (a token a lane: a warp's 32 features of one
        // are 64 or 128 bytes).  A chunk's residual is requested into registers when
        // those of the one before it have been used, across items.
        At next{};
        it_next = next_item(it);
        if (it_next < num_items) {
          next = at_item(it_next);
          const GroupedParams& o = next.i.wt ? pw : p;
          const int f_first = next.i.f0 + (int)rank * 128 + q * 32;
          if (next.has_r && f_first < o.feats) {
            const uint8_t* const first =
                static_cast<const uint8_t*>(o.r) + ((next.i.wt ? (long long)next.i.g * o.sd : 0ll) +
                                                    (long long)next.i.t0 * o.ldr + f_first) * ES;
            for (int c = strm * 32 + lane; c < next.i.valid; c += 32 * kStreams)
              prefetch_l2(first + c * next.r_step);
          }
        }
        const Item& i = t.i;
        // (debug build: what is stored lies inside d)
        if (!dbg_check(i.f0 >= 0 && i.t0 >= 0 && i.valid <= i.width &&
                           i.t0 + i.valid <= (i.wt ? pw.cols : p.rows),
                       kChkEpiStore, w))
          break;
        const int next_c = first_chunk(next_turn(turn));
        int c = first_chunk(turn);
        if (!__all_sync(0xFFFFFFFFu, wait_phase(tfull0 + 8u * acc, aph, w, kWaitEpilogue))) break;
        tc_fence_after_sync();
        if (c >= i.valid) {                      // no chunk of this item is this warp's
          release();
          fetch_first(next, next_c);
        }
        const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * kAccStride;
#pragma unroll 1
        for (; c < i.valid; c += kNext) {
          uint32_t a[kGroupedChunk];
          __syncwarp();
          tmem_load_32cols(tbase + c, a);
          tmem_wait_ld(a);
          const bool last = c + kNext >= i.valid;
          if (last) release();
          if (i.blocks == 0) {                   // (nothing was accumulated)
#pragma unroll
            for (int x = 0; x < kGroupedChunk; ++x) a[x] = 0u;
          }
          // where the next chunk's residual lies
          const long long follow_step = last ? next.r_step : t.r_step;
          const uint8_t* const follow =
              last ? next.r + next_c * follow_step : t.r + (c + kNext) * follow_step;
          const bool follow_r = last ? next.has_r : t.has_r;
          const int follow_left = last ? (next.mine ? next.i.valid - next_c : 0)
                                       : (t.mine ? i.valid - c - kNext : 0);
          const auto half = [&](auto number) {
            constexpr int H = decltype(number)::value;
            float v[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) v[x] = __uint_as_float(a[16 * H + x]) * t.scale;
            if (t.has_r) {
#pragma unroll
              for (int x = 0; x < W; ++x) {
                if constexpr (LEAN == DT_F32) {
                  v[x] += __uint_as_float(res[W * H + x]);
                } else {
                  const uint32_t u = swap_halves(res[W * H + x], odd);
                  const float2 e = LEAN == DT_F16 ? unpack_f16x2(u) : unpack_bf16x2(u);
                  v[2 * x] += e.x;
                  v[2 * x + 1] += e.y;
                }
              }
            }
            if (follow_r) fetch(IntC<W * H>{}, follow + 16 * H * follow_step, follow_step, follow_left - 16 * H);
            uint8_t* p_d = t.d + (c + 16 * H) * t.d_step;
            if (PER == 2 && t.odd_feats) {       // every lane its own feature
              const int left = t.mine ? i.valid - c - 16 * H : 0;
#pragma unroll
              for (int x = 0; x < 16; x += 2, p_d += 2 * t.d_step) {
                const uint32_t u = LEAN == DT_F16 ? pack_f16x2(v[x], v[x + 1]) : pack_bf16x2(v[x], v[x + 1]);
                if (x < left) *reinterpret_cast<uint16_t*>(p_d) = (uint16_t)u;
                if (x + 1 < left) *reinterpret_cast<uint16_t*>(p_d + t.d_step) = (uint16_t)(u >> 16);
              }
            } else {
              const int left = t.mine ? i.valid - c - 16 * H - (int)second : 0;
#pragma unroll
              for (int x = 0; x < W; ++x, p_d += PER * t.d_step) {
                uint32_t o;
                if constexpr (LEAN == DT_F32) o = __float_as_uint(v[x]);
                else o = swap_halves(LEAN == DT_F16 ? pack_f16x2(v[2 * x], v[2 * x + 1])
                                                    : pack_bf16x2(v[2 * x], v[2 * x + 1]), odd);
                if (PER * x < left) *reinterpret_cast<uint32_t*>(p_d) = o;
              }
            }
          };
          half(IntC<0>{});
          half(IntC<1>{});
        }
        t = next;
        if (++acc == kAccStages) { acc = 0; aph ^= 1u; }
      }
    } else {
      const auto bytes = [](int dt) { return dt == DT_F32 ? 4 : 2; };
      const bool r16 = p.r_dt != DT_F32;
      for (int it = first_item; it < num_items; it = next_item(it), turn = next_turn(turn)) {
        const Item i = item_at(it);
        const int f = i.f0 + (int)rank * 128 + q * 32 + lane;
        const bool mine = f < p.feats;
        const bool pairs = !(p.feats & 1) || !__any_sync(0xFFFFFFFFu, f + 1 == p.feats);
        // (debug build: what is stored lies inside d)
        if (!dbg_check(i.f0 >= 0 && i.t0 >= 0 && i.valid <= i.width &&
                           i.t0 + i.valid <= (kWeights ? p.cols : p.rows),
                       kChkEpiStore, w))
          break;
        const auto place = [&](const void* base, long long ld, int dt) {
          uint8_t* const row = static_cast<uint8_t*>(const_cast<void*>(base)) +
                               ((kWeights ? (long long)i.g * p.sd : 0ll) + (long long)i.t0 * ld) * bytes(dt);
          return EpiMatrix{row + (long long)f * bytes(dt),
                           row + (long long)(f & ~1) * bytes(dt) + (odd ? ld * bytes(dt) : 0ll),
                           ld * bytes(dt), dt};
        };
        const EpiMatrix rm = place(p.r, p.ldr, p.r_dt), zm = place(p.z, p.ldz, p.z_dt),
                        dm = place(p.d, p.ldd, p.d_dt);
        float scale = i.blocks ? p.alpha : 0.f, bias = 0.f;
        if constexpr (kRows) {
          if (p.set_scale && i.blocks) scale *= __ldg(p.set_scale + i.e);
        }
        if constexpr (kFull) {
          if (mine && i.e >= 0) {
            const long long at = (long long)i.e * p.feats + f;
            if (p.col_scale && i.blocks) scale *= __ldg(p.col_scale + at);
            if (p.bias) bias = p.bias_dt == DT_F32 ? __ldg(static_cast<const float*>(p.bias) + at)
                               : p.bias_dt == DT_F16
                                   ? __half2float(__ushort_as_half(__ldg(static_cast<const uint16_t*>(p.bias) + at)))
                                   : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p.bias) + at) << 16);
          }
        }
        // Chunks of 32 columns, every other one this warp's; which warp of the two starts
        // alternates, so that items of one chunk are shared out.  The residual of the first
        // two chunks (the first, of 32 bits) and the first's row factors (one a lane) are on their
        // way before the accumulator is waited for, the others two chunks (one) ahead.
        uint32_t res[32];
        float factor = 1.f;
        const auto fetch_32 = [&](int c) {
          epi_load<0>(rm, c, i.valid - c, pairs, mine, odd, res);
          if (c + 16 < i.valid) epi_load<16>(rm, c + 16, i.valid - c - 16, pairs, mine, odd, res);
        };
        const auto fetch_16 = [&](auto from, int c) {
          constexpr int FROM = decltype(from)::value;
          epi_load<FROM>(rm, c, i.valid - c, pairs, mine, odd, res);
          if (c + 16 < i.valid) epi_load<FROM + 8>(rm, c + 16, i.valid - c - 16, pairs, mine, odd, res);
        };
        const auto fetch_factor = [&](int c) {
          if constexpr (kFull) {
            if (p.row_scale && i.blocks > 0)
              factor = c + lane < i.valid ? __ldg(p.row_scale + i.t0 + c + lane) : 1.f;
          }
        };
        const int c_first = first_chunk(turn);
        if (c_first < i.valid) {
          if (p.r) {
            if (r16) {
              fetch_16(IntC<0>{}, c_first);
              if (c_first + kNext < i.valid) fetch_16(IntC<16>{}, c_first + kNext);
            } else {
              fetch_32(c_first);
            }
          }
          fetch_factor(c_first);
        }
        if (!__all_sync(0xFFFFFFFFu, wait_phase(tfull0 + 8u * acc, aph, w, kWaitEpilogue))) break;
        tc_fence_after_sync();
        if (c_first >= i.valid) release();
        const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * kAccStride;
#pragma unroll 1
        for (int c = c_first; c < i.valid; c += kNext) {
          uint32_t a[kGroupedChunk];
          __syncwarp();
          tmem_load_32cols(tbase + c, a);
          tmem_wait_ld(a);
          if (c + kNext >= i.valid) release();
          if (i.blocks == 0) {                     // (nothing was accumulated)
#pragma unroll
            for (int x = 0; x < kGroupedChunk; ++x) a[x] = 0u;
          }
          const auto half = [&](auto from) {
            constexpr int FROM = decltype(from)::value;      // 0, 16
            const int left = i.valid - c - FROM;
            float v[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) v[x] = __uint_as_float(a[FROM + x]) * scale;
            if constexpr (kFull) {
              if (p.row_scale) {
#pragma unroll
                for (int x = 0; x < 16; ++x) v[x] *= __shfl_sync(0xFFFFFFFFu, factor, FROM + x);
              }
              if (p.bias) {
#pragma unroll
                for (int x = 0; x < 16; ++x) v[x] += bias;
              }
              if (p.z) epi_store(zm, c + FROM, left, pairs, mine, odd, v);
              with_activation(p.act, [&](auto act) {
#pragma unroll
                for (int x = 0; x < 16; x += 2) activate2<decltype(act)::value>(v[x], v[x + 1]);
              });
            }
            if (p.r) {
              if (r16) epi_add<FROM / 2>(rm, pairs, odd, res, v);
              else epi_add<FROM>(rm, pairs, odd, res, v);
            }
            epi_store(dm, c + FROM, left, pairs, mine, odd, v);
          };
          half(IntC<0>{});
          if (c + 16 < i.valid) half(IntC<16>{});
          if (c + kNext < i.valid) {
            if (p.r) {
              if (r16) {
#pragma unroll
                for (int x = 0; x < 16; ++x) res[x] = res[16 + x];
                if (c + 2 * kNext < i.valid) fetch_16(IntC<16>{}, c + 2 * kNext);
              } else {
                fetch_32(c + kNext);
              }
            }
            fetch_factor(c + kNext);
          }
        }
        if (++acc == kAccStages) { acc = 0; aph ^= 1u; }
      }
    }
  } else if constexpr (kWeights) {
    // ---------------------------------------------------------- zeroing (weights form)
    int s = 0;
    uint32_t phases = 0;                         // a bit per stage: its tail barrier's phase
    for (int it = first_item; it < num_items; it = next_item(it)) {
      const Item i = item_at(it);
      if (i.wt && i.blocks > 0 && i.mn % UMMA_K != 0) {
        const int at = i.down ? s : (s + i.blocks - 1) % S;
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(tail0 + 8u * at, phases >> at & 1u, w,
                                                      kWaitProducer)))
          break;
        // rows [from, to) of every 128-byte wide atom column
        const int from = i.mn - (i.blocks - 1) * BK, to = (from + UMMA_K - 1) / UMMA_K * UMMA_K;
        uint8_t* const sf = gbase + (f_ring + at * f_stage - base);
        uint8_t* const st = gbase + (t_ring + at * t_stage - base);
        const int boxes = i.width / CG / ATOM_K;
        for (int j = 0; j < F_BOXES + boxes; ++j) {
          uint8_t* const box = j < F_BOXES ? sf + j * MN_ATOM : st + (j - F_BOXES) * MN_ATOM;
          for (int b = from * 128 + lane * 16; b < to * 128; b += 512)
            *reinterpret_cast<uint4*>(box + b) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_all();
        __syncwarp();
        if (rank != 0) {
          if (lane == 0) mbar_arrive_cluster(map_to_rank(peer0 + 8u * at, 0));
        } else {
          if (PAIR && !__all_sync(0xFFFFFFFFu, wait_phase(peer0 + 8u * at, phases >> at & 1u, w,
                                                          kWaitProducer)))
            break;
          if (lane == 0) mbar_arrive(full0 + 8u * at);
        }
        phases ^= 1u << at;
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
