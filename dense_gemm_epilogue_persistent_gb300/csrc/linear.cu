// The linear layer, D = act(alpha row_scale col_scale (A B^T) + bias) + R, and its
// backward pass (include/gemm_gb300.h): argument checks, planning and launches of
// the persistent kernel with the linear epilogue, and the activation-gradient
// kernel.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "activations.cuh"
#include "gemm_gb300.h"
#include "handle.h"
#include "kernels.h"
#include "rows.cuh"
#include "rows_host.h"
#include "split_kernel.cuh"

namespace gb300 {

struct ActGradParams {
  long long lddd, ldz, lddz;
  const void* dd;
  const void* z;                    // null: no activation, dz = dd
  void* dz;                         // or null: only the bias gradient is wanted
  void* dbias;                      // or null
  int M, N;
  int act, dbias_dt;
  int row_split;                    // blocks of a cluster, sharing the rows
};

// dz = dd act'(z) and dbias = its column sums (of the values before dz is
// rounded), 6 bytes and about 25 instructions an element.  A block owns 64
// columns (8 lanes of one vector each) and 1/R of the rows, R the cluster size:
// thread group g of G = THREADS / 8 walks rows first + g, + G, ..., each thread
// copying its own pieces of the next kActDepth rows into its own slots of shared
// memory (16 bytes and the row's end as they lie in memory; before the launch shapes
// were chosen as below, 4096 x 8192 gelu took 39.0 us so and 43.6 with loads into
// registers, two rows at a time, 8192 x 700, whose rows end inside a piece, 13.1 and
// 20.3).  A column's sum is added in a fixed order: a thread's rows, the groups
// through shared memory, the cluster's blocks by its first one.
// (4096 x 8192 gelu: 34.1 us with three rows, 35.1 with two, 34.2 with four; 16384 x
// 4096: 65.5, 67.4, 65.1; 8192 x 700: 13.4, 12.9, 13.4)
constexpr int kActDepth = 3;

template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
act_grad_kernel(const __grid_constant__ ActGradParams p) {
  constexpr int G = THREADS / 8;
  extern __shared__ uint4 act_ring[];    // [kActDepth][dd, z][thread], then
  float(*const part)[64] = reinterpret_cast<float(*)[64]>(act_ring + kActDepth * 2 * THREADS);
  __shared__ float block_part[64];
  constexpr int es = elem_bytes(DT);
  grid_launch_dependents();
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int R = p.row_split, rank = blockIdx.x % R, strip = blockIdx.x / R;
  const int c = strip * 64 + lane * kVec;
  const int share = (p.M + R - 1) / R;
  const long long first = (long long)rank * share;
  const long long last = min((long long)p.M, first + share);
  float acc[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
  grid_dependency_wait();
  if (c < p.N) {
    const uint8_t* const dd = static_cast<const uint8_t*>(p.dd);
    const uint8_t* const zz = static_cast<const uint8_t*>(p.z);
    with_activation(p.act, [&](auto a) {
      constexpr int ACT = decltype(a)::value;
      const int bytes = min(kVec, p.N - c) * es;
      const uint32_t ring = smem_u32(act_ring) + threadIdx.x * 16;
      auto request = [&](long long row, int slot) {
        if (row < last) {
          const uint32_t at = ring + slot * (2 * THREADS * 16);
          copy16_async(at, dd + (row * p.lddd + c) * es, bytes);
          if constexpr (ACT != ACT_NONE)
            copy16_async(at + THREADS * 16, zz + (row * p.ldz + c) * es, bytes);
        }
        copy_commit();
      };
#pragma unroll
      for (int s = 0; s < kActDepth; ++s) request(first + group + s * G, s);
      int slot = 0;
      for (long long row = first + group; row < last; row += G) {
        copy_wait(kActDepth - 1);
        const uint4* const at = act_ring + slot * (2 * THREADS) + threadIdx.x;
        float g[kVec];
        unpack<DT>(RawVec<DT>{{at[0]}}, g);
        if constexpr (ACT != ACT_NONE) {
          float z[kVec];
          unpack<DT>(RawVec<DT>{{at[THREADS]}}, z);
#pragma unroll
          for (int i = 0; i < kVec; i += 2)
            unpair(mul2(pair(g[i], g[i + 1]), activate_grad2<ACT>(z[i], z[i + 1])), g[i], g[i + 1]);
        }
        if (p.dz) store_vec(static_cast<uint8_t*>(p.dz) + row * p.lddz * es, DT, c, p.N, g);
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[i] += g[i];
        request(row + kActDepth * G, slot);       // (into the slot just read)
        if (++slot == kActDepth) slot = 0;
      }
    });
  }
  if (!p.dbias) return;                  // (the whole grid)
#pragma unroll
  for (int i = 0; i < kVec; ++i) part[group][lane * kVec + i] = acc[i];
  __syncthreads();
  // 4 threads a column take a quarter of the groups each, added in lane order.
  if (threadIdx.x < 256) {
    const int col = threadIdx.x >> 2, quarter = threadIdx.x & 3;
    float s = 0.f;
#pragma unroll 8
    for (int i = quarter * (G / 4); i < (quarter + 1) * (G / 4); ++i) s += part[i][col];
    s += __shfl_down_sync(0xFFFFFFFFu, s, 1);
    s += __shfl_down_sync(0xFFFFFFFFu, s, 2);
    if (quarter == 0) block_part[col] = s;
  }
  if (R > 1) cluster_sync_all(); else __syncthreads();
  const int col = strip * 64 + (int)threadIdx.x;
  if (rank == 0 && threadIdx.x < 64 && col < p.N) {
    float s = block_part[threadIdx.x];
    for (int r = 1; r < R; ++r)
      s += load_cluster_f32(map_to_rank(smem_u32(&block_part[threadIdx.x]), (uint32_t)r));
    store_elem(p.dbias, col, p.dbias_dt, s);
  }
  if (R > 1) cluster_sync_all();         // the first block has read the others' sums
}

}  // namespace gb300

namespace {

using namespace gb300host;

bool is_activation(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }

// Sizes the kernels index with 32 bits: what they add to an index on the way to its
// bound (the rest of the last tile, whose width need not divide 2^31; a vector's
// end; a cluster's shares of the rows) stays below 2^31.
bool is_extent(int64_t v) { return v >= 0 && v <= INT32_MAX - 8192; }
// Tensor-map strides below 2^40 bytes.
bool map_ok(int64_t ld, int64_t rows, int dt) {
  return (double)ld * dtype_bytes(dt) * (double)rows < 1099511627776.0;
}

// One A or B operand: `inner` contiguous elements a row, `rows` rows.
gemm_status_t check_operand(const void* p, int64_t ld, int64_t inner, int64_t rows, int dt) {
  GB300_CHECK(check_matrix(p, ld, inner, dt));
  return map_ok(ld, rows, dt) ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

gemm_status_t check_linear(const gemm_linear_t& p) {
  if (!is_extent(p.M) || !is_extent(p.N) || !is_extent(p.K)) return GEMM_ERR_INVALID_ARG;
  if (!is_layout(p.layoutA) || !is_layout(p.layoutB) || !is_activation(p.activation))
    return GEMM_ERR_INVALID_ARG;
  if (!is_ab_type(p.a_type) || !is_ab_type(p.b_type) ||
      (p.a_type != p.b_type && !(is_fp8(p.a_type) && is_fp8(p.b_type))))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (p.a_type == GEMM_TF32 && (p.layoutA != GEMM_K_MAJOR || p.layoutB != GEMM_K_MAJOR))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (!is_epi_type(p.d_type) || (p.bias && !is_epi_type(p.bias_type)) ||
      (p.R && !is_epi_type(p.r_type)) || (p.Z && !is_epi_type(p.z_type)))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (p.M == 0 || p.N == 0) return GEMM_OK;
  if (cdiv(p.M, 128) * cdiv(p.N, 128) > INT32_MAX / 2) return GEMM_ERR_INVALID_ARG;
  GB300_CHECK(check_operand(p.D, p.ldd, p.N, p.M, p.d_type));
  if (p.R) GB300_CHECK(check_operand(p.R, p.ldr, p.N, p.M, p.r_type));
  if (p.Z) GB300_CHECK(check_operand(p.Z, p.ldz, p.N, p.M, p.z_type));
  if (p.K > 0) {
    const bool am = p.layoutA == GEMM_MN_MAJOR, bm = p.layoutB == GEMM_MN_MAJOR;
    GB300_CHECK(check_operand(p.A, p.lda, am ? p.M : p.K, am ? p.K : p.M, p.a_type));
    GB300_CHECK(check_operand(p.B, p.ldb, bm ? p.N : p.K, bm ? p.K : p.N, p.b_type));
  }
  if (!aligned_to(p.row_scale, 4) || !aligned_to(p.col_scale, 4) ||
      (p.bias && !aligned_to(p.bias, dtype_bytes(p.bias_type))))
    return GEMM_ERR_MISALIGNED;
  // in place: element for element only; nothing else may share an output
  if (p.R == p.D && (p.r_type != p.d_type || p.ldr != p.ldd)) return GEMM_ERR_INVALID_ARG;
  if (p.Z && (p.Z == p.D || p.Z == p.R)) return GEMM_ERR_INVALID_ARG;
  if (p.K > 0 && (p.D == p.A || p.D == p.B || (p.Z && (p.Z == p.A || p.Z == p.B))))
    return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

// The planner's view of the call: the residual as C, the pre-activation as Y.
gemm_problem_t as_problem(const gemm_linear_t& p) {
  gemm_problem_t g{};
  g.M = p.M; g.N = p.N; g.K = p.K; g.L = 1;
  g.A = p.A; g.lda = p.lda; g.layoutA = p.layoutA;
  g.B = p.B; g.ldb = p.ldb; g.layoutB = p.layoutB;
  g.C = p.R; g.D = p.D; g.Y = p.Z;
  g.alpha = p.alpha;
  g.beta = p.R ? 1.f : 0.f;
  g.dtypes.ab = p.a_type;
  g.dtypes.b = p.b_type == p.a_type ? GEMM_F32 : p.b_type;
  g.dtypes.c = p.R ? p.r_type : GEMM_F32;
  g.dtypes.d = p.d_type;
  g.dtypes.x = GEMM_F32;
  g.dtypes.y = p.Z ? p.z_type : GEMM_F32;
  g.dtypes.cdxy_major = GEMM_K_MAJOR;
  g.dtypes.acc = GEMM_F32;
  return g;
}

// Time the epilogue's arithmetic adds to a chunk, in the cost model's units
// (gemm_api.cu, tile_cost).
double activation_cost(int act) {
  switch (act) {
    case GEMM_ACT_GELU: return 1.6;
    case GEMM_ACT_GELU_TANH: return 1.0;
    case GEMM_ACT_SILU: return 0.9;
    default: return 0.2;
  }
}

// A 16-bit product with nothing but alpha and a residual behind it: the kernel of
// two products runs it without a second one, whose epilogue has no column
// vectors and activations (4096 x 4096 x 512 bf16 20.6 us, 23.5 by the full one; 2048 x
// 4096 x 1024 18.5, 19.4; 8192 x 8192 x 1024 81, 89; with a residual 30.6, 31.7; 8192^3 the
// same).
bool is_plain(const gemm_linear_t& p) {
  return (p.a_type == GEMM_F16 || p.a_type == GEMM_BF16) && p.activation == GEMM_ACT_NONE &&
         !p.row_scale && !p.col_scale && !p.bias && !p.Z && p.K > 0;
}

// Plan a checked call on the persistent kernel (h->mu held); *cost receives the
// cost model's figure.
gemm_status_t plan_persistent(gemm_handle* h, const gemm_linear_t& p, LinearPlan& out,
                              double* cost) {
  const gemm_problem_t g = as_problem(p);
  gemm_config_t& cfg = out.cfg;
  GB300_CHECK(plan_valid(g, h->sm_count, h->smem_optin, h->forced ? &h->forced_cfg : nullptr, &cfg,
                         h->clusters_by_size, false,
                         EpilogueExtra{true, (int)gb300::kLinearSmem, activation_cost(p.activation)},
                         cost));
  if (cfg.cluster_m != 1 || cfg.cluster_n != 1) return GEMM_ERR_UNSUPPORTED_CONFIG;
  const int es = dtype_bytes(p.a_type);
  const int ka = gb300::k_atoms(cfg.cta_group, cfg.tile_n);
  out.plain = is_plain(p);
  out.kern = gb300::linear_kernel_for(es, cfg.cta_group, ka, cfg.epi_warps, out.plain ? 2 : 1);
  if (!out.kern) return GEMM_ERR_UNSUPPORTED_CONFIG;
  VariantState& vs = out.plain ? h->pair_variants[cfg.cta_group - 1][ka - 1][cfg.epi_warps - 1]
                               : h->linear_variants[es == 2 ? 0 : es == 1 ? 1 : 2]
                                                   [cfg.cta_group - 1][ka - 1][cfg.epi_warps - 1];
  int resident = 0;
  GB300_CHECK(resident_kernel_clusters(h, vs, out.kern, cfg, cfg.cta_group, &resident));
  cfg.grid_ctas = (int)std::min<int64_t>(cfg.tiles + cfg.tail_split, resident) * cfg.cta_group;
  return GEMM_OK;
}

// A launch's place beside another that it does not depend on (EpiParams).
enum Place { kAlone, kFirstOfTwo, kSecondOfTwo };

// A call's tensor maps (A, B, C, X, D, Y) and parameters for the persistent kernel.
gemm_status_t prepare_persistent(gemm_handle* h, const gemm_linear_t& p, const gemm_config_t& cfg,
                                 CUtensorMap (&maps)[6], KernelParams& kp) {
  std::memset(maps, 0, sizeof(maps));
  const bool a_mn = p.layoutA == GEMM_MN_MAJOR, b_mn = p.layoutB == GEMM_MN_MAJOR;
  if (p.K > 0 &&
      (!encode_operand(h->encode, &maps[0], p.A, p.a_type, p.M, p.K, 1, p.lda, a_mn, 128,
                       cfg.tile_k) ||
       !encode_operand(h->encode, &maps[1], p.B, p.b_type, p.N, p.K, 1, p.ldb, b_mn,
                       cfg.tile_n / cfg.cta_group, cfg.tile_k)))
    return GEMM_ERR_CUDA;
  // D and Z as far as their rows' whole 16-byte pieces (a row without one is
  // not stored through its map).
  const auto stored = [&](gemm_dtype_t t) {
    const int64_t piece = 16 / dtype_bytes(t);
    return p.N < piece ? p.N : p.N - p.N % piece;
  };
  if ((p.R && !encode_epi(h->encode, &maps[2], p.R, p.r_type, p.M, p.N, 1, false, p.ldr)) ||
      !encode_epi(h->encode, &maps[4], p.D, p.d_type, p.M, stored(p.d_type), 1, false, p.ldd) ||
      (p.Z &&
       !encode_epi(h->encode, &maps[5], p.Z, p.z_type, p.M, stored(p.z_type), 1, false, p.ldz)))
    return GEMM_ERR_CUDA;

  kp.M = (int)p.M; kp.N = (int)p.N; kp.K = (int)p.K; kp.L = 1;
  kp.bn = cfg.tile_n;
  kp.tiles_m = (int)cdiv(p.M, cfg.tile_m);
  kp.tiles_n = (int)cdiv(p.N, cfg.tile_n);
  kp.num_tiles = (int)cfg.tiles;
  kp.k_blocks = (int)cdiv(p.K, cfg.tile_k);
  kp.group_m = cfg.group_m;
  kp.stages = cfg.stages;
  kp.a_mn_major = a_mn;
  kp.b_mn_major = b_mn;
  kp.idesc = make_idesc(p.a_type, p.b_type, false, cfg.cta_group, cfg.tile_n, a_mn, b_mn);
  kp.idesc_half = make_idesc(p.a_type, p.b_type, false, cfg.cta_group, cfg.tile_n / 2, a_mn, b_mn);
  kp.split_start = (int)(cfg.tiles - cfg.tail_split);
  kp.num_items = (int)(cfg.tiles + cfg.tail_split);
  kp.l2_hints = (uint32_t)cfg.l2_hints;
  kp.epi_wait_ns = (uint32_t)cfg.epi_wait_ns;
  kp.inject_stall = cfg.inject_stall;
  kp.k_alternate = 1;
  kp.status = h->d_status;
  kp.timeout_ns = h->timeout_ns;
  kp.stats = h->d_stats;
  kp.epi.c_dt = p.R ? p.r_type : GEMM_F32;
  kp.epi.d_dt = p.d_type;
  kp.epi.x_dt = GEMM_F32;
  kp.epi.y_dt = p.Z ? p.z_type : GEMM_F32;
  kp.epi.read_c = p.R != nullptr;
  kp.epi.write_y = p.Z != nullptr;
  kp.epi.alpha = p.alpha;
  kp.epi.slots = cfg.epi_slots;
  const int sub = 128 * gb300::kEpiChunk;
  kp.epi.cd_bytes = (uint32_t)(sub * std::max(dtype_bytes(p.d_type), p.R ? dtype_bytes(p.r_type) : 0));
  kp.epi.xy_bytes = (uint32_t)cfg.epi_slot_bytes - kp.epi.cd_bytes;
  kp.epi.row_scale = p.row_scale;
  kp.epi.col_scale = p.col_scale;
  kp.epi.bias = p.bias;
  kp.epi.bias_dt = p.bias_type;
  kp.epi.act = p.activation;
  kp.epi.d_ptr = p.D; kp.epi.ldd = p.ldd;
  kp.epi.d_ragged = (p.N * dtype_bytes(p.d_type)) % 16 != 0;
  if (p.Z) {
    kp.epi.y_ptr = p.Z; kp.epi.ldy = p.ldz;
    kp.epi.y_ragged = (p.N * dtype_bytes(p.z_type)) % 16 != 0;
  }
  return GEMM_OK;
}

gemm_status_t launch_persistent(const gemm_config_t& cfg, const void* kern, void** args,
                                struct CUstream_st* stream) {
  cudaLaunchConfig_t lc{};
  cudaLaunchAttribute attr[2];
  lc.gridDim = dim3((unsigned)cfg.grid_ctas);
  lc.blockDim = dim3((unsigned)gb300::threads_for(cfg.epi_warps));
  lc.dynamicSmemBytes = (size_t)cfg.smem_bytes;
  lc.stream = reinterpret_cast<cudaStream_t>(stream);
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cfg.cta_group;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  if (cudaLaunchKernelExC(&lc, kern, args) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

// Enqueue a call on the persistent kernel by its plan.
gemm_status_t run_persistent(gemm_handle* h, const gemm_linear_t& p, const LinearPlan& plan,
                             Place place, struct CUstream_st* stream) {
  CUtensorMap maps[6];
  gb300::PairParams kp{};              // (read as KernelParams by the other kernels)
  GB300_CHECK(prepare_persistent(h, p, plan.cfg, maps, kp));
  kp.first_items = kp.num_items;
  kp.epi.trigger_late = place == kFirstOfTwo;
  kp.epi.wait_late = place == kSecondOfTwo;
  void* args[7] = {&maps[0], &maps[1], &maps[2], &maps[3], &maps[4], &maps[5], &kp};
  return launch_persistent(plan.cfg, plan.kern, args, stream);
}

// The ring, its barriers and the alignment; the last stage's matrix operand,
// 128 rows whatever `feats`, has to lie inside.
int split_smem(int bn, int feats, int ka, int stages) {
  const int tail = std::max(0, (128 - feats) * 128 - stages * ka * bn * 128);
  return stages * ka * (feats + bn) * 128 + tail + (int)gb300::kSplitBarBytes + 1024;
}

// Dynamic shared memory of its CTAs: 113 KB, half of an SM's 228 KB less the
// 1 KB the system takes for each.
constexpr int kSplitSmem = 113 * 1024;

// Whether the kernel can run `p` with such tiles, and the plan.  K is split
// into at most one k-block per CTA; MN-major tokens are staged in whole atoms.
bool plan_split(const gemm_linear_t& p, int bn, int feats, int split, SplitPlan* out) {
  const int es = dtype_bytes(p.a_type);
  const int64_t k_blocks = cdiv(p.K, 128 / es);
  if (p.K == 0 || bn < 16 || bn > 128 || bn % 16 != 0 || split < 1 || split > 8 ||
      feats < 8 || feats > 128 || feats % 8 != 0 || split > k_blocks)
    return false;
  if (p.layoutB == GEMM_MN_MAJOR && feats != 128) return false;
  if (p.layoutA == GEMM_MN_MAJOR && bn % (128 / es) != 0) return false;
  out->bn = bn;
  out->feats = feats;
  out->split = split;
  out->tiles_m = cdiv(p.M, bn);
  out->tiles_n = cdiv(p.N, feats);
  // Two CTAs fit an SM, so that the next launch's set-up overlaps the end of
  // this one; three do not, and neither does one beside a CTA of the
  // persistent kernel (half an SM's shared memory and 1 KB at least): whatever
  // shares an SM then has its tensor memory (128 columns at most each) at once,
  // and no cluster waits for one that waits for it.
  out->smem = kSplitSmem;
  out->ka = split_smem(bn, feats, 2, 3) <= out->smem ? 2 : 1;
  out->stages = 0;
  while (out->stages < gb300::kSplitMaxStages &&
         split_smem(bn, feats, out->ka, out->stages + 1) <= out->smem)
    ++out->stages;
  // The exchange takes place in the ring.
  const int own = (int)cdiv(cdiv(bn, split), 4) * 4;
  if (out->stages < 2 || (split > 1 && split * own * 512 > out->stages * out->ka * (feats + bn) * 128))
    return false;
  return out->tiles_m * out->tiles_n * split <= INT32_MAX;
}

// What gemm_last_config reports of a split-K launch.
gemm_config_t config_of(const SplitPlan& s, int es) {
  gemm_config_t c{};
  c.cta_group = 1;
  c.tile_m = s.feats;
  c.tile_n = s.bn;
  c.tile_k = 128 / es * s.ka;
  c.stages = s.stages;
  c.acc_stages = 1;
  c.ring_bytes = s.stages * s.ka * (s.feats + s.bn) * 128;
  c.smem_bytes = s.smem;
  c.tiles = s.tiles_m * s.tiles_n;
  c.grid_ctas = (int)(c.tiles * s.split);
  c.epi_warps = s.bn <= 16 ? 1 : 2;
  c.split_k = s.split;
  return c;
}

gemm_status_t run_split(gemm_handle* h, const gemm_linear_t& p, const LinearPlan& plan,
                        Place place, struct CUstream_st* stream) {
  const SplitPlan& s = plan.s;
  const int es = dtype_bytes(p.a_type);
  const bool a_mn = p.layoutA == GEMM_MN_MAJOR, b_mn = p.layoutB == GEMM_MN_MAJOR;
  CUtensorMap feat, tok;
  if (!encode_operand(h->encode, &feat, p.B, p.b_type, p.N, p.K, 1, p.ldb, b_mn, s.feats,
                      128 / es) ||
      !encode_operand(h->encode, &tok, p.A, p.a_type, p.M, p.K, 1, p.lda, a_mn, s.bn, 128 / es))
    return GEMM_ERR_CUDA;
  gb300::SplitParams k{};
  k.M = (int)p.M; k.N = (int)p.N;
  k.bn = s.bn;
  k.feats = s.feats;
  k.ka = s.ka;
  k.tiles_m = (int)s.tiles_m;
  k.split = s.split;
  k.own = (int)cdiv(cdiv(s.bn, s.split), 4) * 4;
  k.k_blocks = (int)cdiv(p.K, 128 / es);
  k.stages = s.stages;
  k.feat_mn = b_mn;
  k.tok_mn = a_mn;
  k.idesc = make_idesc(p.b_type, p.a_type, false, 1, s.bn, b_mn, a_mn);
  k.tmem_cols = 32;
  while ((int)k.tmem_cols < s.bn) k.tmem_cols *= 2;
  k.status = h->d_status;
  k.timeout_ns = h->timeout_ns;
  k.alpha = p.alpha;
  k.row_scale = p.row_scale;
  k.col_scale = p.col_scale;
  k.bias = p.bias; k.bias_dt = p.bias_type;
  k.r = p.R; k.ldr = p.ldr; k.r_dt = p.r_type;
  k.z = p.Z; k.ldz = p.ldz; k.z_dt = p.z_type;
  k.d = p.D; k.ldd = p.ldd; k.d_dt = p.d_type;
  k.act = p.activation;
  k.inject_stall = plan.cfg.inject_stall;
  k.trigger_late = place == kFirstOfTwo;
  k.wait_late = place == kSecondOfTwo;
  cudaLaunchConfig_t lc{};
  cudaLaunchAttribute attr[2];
  lc.gridDim = dim3((unsigned)(s.tiles_m * s.tiles_n * s.split));
  lc.blockDim = dim3((unsigned)gb300::threads_for(plan.cfg.epi_warps));
  lc.dynamicSmemBytes = (size_t)s.smem;
  lc.stream = reinterpret_cast<cudaStream_t>(stream);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)s.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = s.split > 1 ? 2 : 1;
  void* args[3] = {&feat, &tok, &k};
  if (cudaLaunchKernelExC(&lc, plan.kern, args) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

// Clusters of `split` CTAs the device holds at one CTA an SM (what the cluster
// size leaves over in each GPC taken off), asked for once per size.  (The
// occupancy calculator counts one CTA an SM for this kernel; two are resident, as
// start and end times of consecutive launches' blocks show.)
int split_clusters(gemm_handle* h, int split) {
  int& n = h->split_clusters[split];
  if (n > 0) return n;
  const void* kern = gb300::split_kernel_for(2);
  cudaLaunchConfig_t lc{};
  cudaLaunchAttribute attr[1];
  lc.gridDim = dim3((unsigned)(split * 2 * h->sm_count));
  lc.blockDim = dim3((unsigned)gb300::kSplitThreads);
  lc.dynamicSmemBytes = (size_t)kSplitSmem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (raise_smem(h, kern) != GEMM_OK ||
      cudaOccupancyMaxActiveClusters(&n, kern, &lc) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = std::max(1, h->sm_count / split);
  }
  return n;
}

// The split-K kernel's tiles where the call chooses: all features of an MMA,
// the tokens cut evenly into tiles of at most 128 (whole atoms where they are
// MN-major), and as many CTAs a tile, with two k-blocks each, as leave every
// tile's cluster resident, at 2.2 times the calculator's clusters (48 x 5000 x 4096
// E4M3, 40 tiles: 8.8 us with 6, 9.8 with 5; with 7 some clusters wait for others to
// end, 13.8; 1 x 8192 x 8192 bf16, 64 tiles: 21.1 with 4, 23.7 with 3; 1 x 4096 x 4096,
// 32 tiles: 9.3 with 8, 9.8 with 6).
bool choose_split(gemm_handle* h, const gemm_linear_t& p, SplitPlan* out) {
  const int es = dtype_bytes(p.a_type);
  const int64_t per_tile = cdiv(p.M, cdiv(p.M, 128));
  int bn = (int)cdiv(per_tile, 16) * 16;
  if (p.layoutA == GEMM_MN_MAJOR) bn = (int)cdiv(bn, 128 / es) * (128 / es);
  if (bn > 128 || p.K == 0) return false;
  const int64_t tiles = cdiv(p.M, bn) * cdiv(p.N, 128);
  if (tiles > 2 * (int64_t)h->sm_count) return false;
  int split = (int)std::max<int64_t>(1, std::min<int64_t>(8, cdiv(p.K, 128 / es) / 2));
  while (split > 1 && 10 * tiles > 22 * (int64_t)split_clusters(h, split)) --split;
  return plan_split(p, bn, 128, split, out);
}

// Which kernel: estimated microseconds of both, linear fits to 200 problems on
// GB300 (1 to 1024 tokens, 512 to 8192 features and inner sizes, bf16 and E4M3, every
// layout).  Choosing by them costs 0.1 % over the faster kernel on average and 5 %
// at worst.  For instance (split-K, persistent): 1 x 4096 x 4096 bf16 9.4, 32.6 us;
// 64 x 4096 x 4096 11.4, 15.6; 128 x 4096 x 4096 16.7, 15.7; 256 x 1024 x 8192 16.4,
// 22.3; 512 x 512 x 512 8.1, 5.7.
double split_us(const gemm_linear_t& p, const SplitPlan& s) {
  const int es = dtype_bytes(p.a_type);
  const double weights = (double)p.N * (double)p.K * es / 6.3e6;       // us at 6.3 TB/s
  const double tokens = (double)p.M * (double)p.K * es * (double)s.tiles_n / 6.3e6;
  const double k_blocks = (double)cdiv(p.K, 128 / es) / s.split;
  const double own = (double)cdiv(cdiv(s.bn, s.split), 4) * 4;
  return 3.41 + 0.141 * k_blocks + 0.0525 * own + (s.split > 1 ? 0.032 * s.bn : 0.0) +
         0.592 * weights + 0.582 * tokens;
}

double persistent_us(const gemm_linear_t& p, double cost) {
  const double weights = (double)p.N * (double)p.K * dtype_bytes(p.a_type) / 6.3e6;
  return 1.59 + 0.333 * cost + 0.498 * weights;
}

// Plan a checked call (h->mu held): as forced, or the faster kernel.
gemm_status_t plan_linear(gemm_handle* h, const gemm_linear_t& p, LinearPlan& out) {
  const int es = dtype_bytes(p.a_type);
  const gemm_config_t& f = h->forced_cfg;
  double cost = 0.0;
  if (h->forced && f.split_k > 0) {
    if (!plan_split(p, f.tile_n ? f.tile_n : 64, f.tile_m ? f.tile_m : 128, f.split_k, &out.s))
      return GEMM_ERR_UNSUPPORTED_CONFIG;
    out.split = true;
  } else {
    GB300_CHECK(plan_persistent(h, p, out, &cost));
    out.us = persistent_us(p, cost);
    out.split = false;
    if (!h->forced && choose_split(h, p, &out.s)) {
      const double us = split_us(p, out.s);
      out.split = us < out.us;
      out.us = std::min(us, out.us);
    }
  }
  if (out.split) {
    out.kern = gb300::split_kernel_for(es);
    GB300_CHECK(raise_smem(h, out.kern));
    out.cfg = config_of(out.s, es);
    out.cfg.inject_stall = h->forced && f.inject_stall ? 1 : 0;
  }
  return GEMM_OK;
}

// The plan of a checked call that is not empty (h->mu held): one of the latest, or made
// now.
gemm_status_t find_plan(gemm_handle* h, const gemm_linear_t& p, LinearPlan& out) {
  LinearKey key;
  std::memset(&key, 0, sizeof(key));           // padding included: keys compare bytewise
  key.M = p.M; key.N = p.N; key.K = p.K;
  key.config_gen = h->config_gen;
  key.a_type = p.a_type; key.b_type = p.b_type; key.d_type = p.d_type;
  key.r_type = p.R ? p.r_type : 0; key.z_type = p.Z ? p.z_type : 0;
  key.layoutA = p.layoutA; key.layoutB = p.layoutB;
  key.activation = p.activation;
  key.has_r = p.R != nullptr; key.has_z = p.Z != nullptr;
  key.plain = is_plain(p);
  LinearPlan* plan = nullptr;
  for (LinearPlan& c : h->linear_plans)
    if (c.valid && std::memcmp(&c.key, &key, sizeof(key)) == 0) { plan = &c; break; }
  if (!plan) {
    plan = &h->linear_plans[h->linear_next];
    plan->valid = false;
    GB300_CHECK(plan_linear(h, p, *plan));
    plan->key = key;
    plan->valid = true;
    h->linear_next = (h->linear_next + 1) % kLinearPlans;
  }
  out = *plan;
  return GEMM_OK;
}

// Enqueue a call by its plan (h->mu held).
gemm_status_t run_planned(gemm_handle* h, const gemm_linear_t& p, const LinearPlan& plan,
                          Place place, struct CUstream_st* stream) {
  h->last = plan.cfg;
  return plan.split ? run_split(h, p, plan, place, stream)
                    : run_persistent(h, p, plan, place, stream);
}

// Microseconds of one item of one of two products in one launch, beside the
// launch's own.  `bytes`: of C and D an element.  The constants here and in
// plan_pair are fitted on GB300 to 61 problems (256 to 8192 tokens, 364 to 8192
// features and inner sizes; db in bf16, or in fp32 and added to) x 28 variants: the
// choice is 0.5 % over the fastest on average and 9 % at worst.
double pair_item(const gemm_config_t& c, int64_t k_blocks, int bytes) {
  const double w = c.tile_n / 256.0;
  double per_kb = c.cta_group == 1 ? 0.250 * w + 0.082 : 0.280 * w + 0.020;
  per_kb *= 1.0 + 0.281 * std::max(0.0, 180.0 - c.ring_bytes / 1024.0) / 64.0;
  const double fixed = c.cta_group == 1 ? 0.185 + 1.390 * w : 1.671 + 0.293 * w;
  return (double)k_blocks * per_kb + fixed + (c.epi_warps == 1 ? 2.177 * w : 0.0) +
         0.388 * w * std::max(0, bytes - 2);
}

// The longest cluster's time, when `first` items of one product, then `second` of the
// other (the last `halves` of them half-width) are dealt to `clusters` clusters,
// `lead` of the second's ahead to those from lead_from on (PairParams).
double pair_time(int64_t first, int64_t second, int64_t halves, int64_t lead, int64_t lead_from,
                 int64_t clusters, double first_us, double second_us) {
  double longest = 0.0;
  for (int64_t c = 0; c < clusters; ++c) {
    const int64_t n1 = c < first ? cdiv(first - c, clusters) : 0;
    const int64_t rest = second - lead;
    const int64_t n2 = c < rest ? cdiv(rest - c, clusters) : 0;
    const int64_t ahead = c >= lead_from ? lead / (clusters - lead_from) : 0;
    double t = (double)n1 * first_us + (double)(n2 + ahead) * second_us;
    if (n2 > 0 && c + (n2 - 1) * clusters >= rest - halves) t -= 0.3 * second_us;
    longest = std::max(longest, t);
  }
  return longest;
}

// Plan the two gradients as one launch (h->mu held): both on the persistent
// kernel with a common tile, the one with more k-blocks a tile first, the last
// round in half-width items where that fits.  One launch wherever each would
// take the persistent kernel anyway (1001 x 2003 x 1501 fp16 17.4 us, 26.4 as two;
// 600 x 600 x 600 7.2, 13.4; 3000 x 5000 x 4096 bf16 142, 164, with db in fp32 and added to
// 154, 205): a launch's start and end, and the last wave's idle SMs, are paid once.
// Where one would take split-K, by the estimates (5000 x 768 x 768 bf16 19.9 us in one,
// 28.4; 128 x 8192 x 512 27.3, 20.4).  Fewer than 128 tokens stay two launches: db's
// items are then one or two k-blocks long, which the estimate does not hold for
// (64 x 4096 x 4096: 36 as it would choose, 31; 1 x 8192 x 2048: 43, 30).
gemm_status_t plan_pair(gemm_handle* h, const gemm_linear_t& da, const gemm_linear_t& db,
                        PairPlan& out) {
  out.one = false;
  const gemm_config_t* const forced = h->forced ? &h->forced_cfg : nullptr;
  if (da.M < 128 || (forced && forced->split_k > 0)) return GEMM_OK;
  bool any_split = false;
  double alone = 0.0;
  for (const gemm_linear_t* p : {&da, &db}) {
    LinearPlan plan;
    GB300_CHECK(plan_linear(h, *p, plan));
    any_split = any_split || plan.split;
    alone += plan.us;
  }
  out.db_first = db.K > da.K;
  const gemm_linear_t& first = out.db_first ? db : da;
  const gemm_linear_t& second = out.db_first ? da : db;
  // The common ring and slots: db's operands ask for more than da's (both
  // MN-major); the wider output type, and db itself where it is added to.
  gemm_linear_t both = db;
  if (dtype_bytes(da.d_type) > dtype_bytes(db.d_type)) both.d_type = da.d_type;
  const EpilogueExtra extra{true, (int)gb300::kLinearSmem, activation_cost(GEMM_ACT_NONE)};
  double best = 0.0;
  for (int cg : {2, 1})
    for (int bn = 256; bn >= 64; bn -= 32)
      for (int epw : {2, 1}) {
        gemm_config_t f = forced ? *forced : gemm_config_t{};
        if ((f.cta_group && f.cta_group != cg) || (f.tile_n && f.tile_n != bn) ||
            (f.epi_warps && f.epi_warps != epw))
          continue;
        const bool may_split = f.tail_split != 1 && (bn / 2) % gb300::kEpiChunk == 0 &&
                               (bn / cg / 2) % 64 == 0;
        f.cta_group = cg;
        f.tile_n = bn;
        f.epi_warps = epw;
        f.tail_split = 1;
        gemm_config_t c, each[2];
        const auto plan = [&](const gemm_linear_t& p, gemm_config_t* o) {
          return plan_valid(as_problem(p), h->sm_count, h->smem_optin, &f, o, h->clusters_by_size,
                            false, extra) == GEMM_OK;
        };
        if (!plan(both, &c) || !plan(first, &each[0]) || !plan(second, &each[1]) ||
            c.cluster_m != 1 || c.cluster_n != 1)
          continue;
        const int ka = gb300::k_atoms(cg, bn);
        const void* kern = gb300::linear_kernel_for(2, cg, ka, epw, 2);
        int resident = 0;
        GB300_CHECK(resident_kernel_clusters(h, h->pair_variants[cg - 1][ka - 1][epw - 1], kern, c,
                                             cg, &resident));
        double us[2];
        for (int i = 0; i < 2; ++i) {
          const gemm_linear_t& p = i ? second : first;
          us[i] = pair_item(c, cdiv(p.K, 64),
                            dtype_bytes(p.d_type) + (p.R ? dtype_bytes(p.r_type) : 0));
        }
        const int64_t n1 = each[0].tiles, n2 = each[1].tiles;
        if (n1 + n2 > INT32_MAX / 2) continue;
        // All SMs' operand loads at the 16.3 TB/s that they come to together.
        const double l2_us = (double)(n1 * cdiv(first.K, 64) + n2 * cdiv(second.K, 64)) *
                             (double)(cg * 128 + bn) * 128.0 / 16.3e6;
        const int64_t clusters = std::min<int64_t>(n1 + n2, resident);
        // Rounds of the second's items for the clusters with one of the first's
        // less; the last round of the rest in half-width items or not.
        const int64_t from = n1 % clusters;
        const int64_t most =
            from ? std::min<int64_t>(n2 / (clusters - from), (int64_t)(us[0] / us[1]) + 1) : 0;
        for (int64_t rounds = 0; rounds <= most; rounds += 1 + most / 32) {
          const int64_t lead = rounds * (clusters - from), rem = (n2 - lead) % clusters;
          for (const int64_t split : {(int64_t)0, may_split && 2 * rem <= clusters ? rem : 0}) {
            const double longest =
                pair_time(n1, n2 + split, 2 * split, lead, from, clusters, us[0], us[1]);
            const double t = std::max(longest, l2_us) + 0.01 * longest;
            if (out.one && t >= best) continue;
            best = t;
            out.one = true;
            out.kern = kern;
            out.lead_items = (int)lead;
            out.lead_from = (int)from;
            out.cfg = c;
            out.cfg.tiles = n1 + n2;
            out.cfg.tail_split = (int)split;
            out.cfg.grid_ctas = (int)clusters * cg;
            for (int i = 0; i < 2; ++i) {
              gemm_config_t& o = out.each[out.db_first ? 1 - i : i];
              o = out.cfg;
              o.tiles = each[i].tiles;
              o.group_m = each[i].group_m;
              o.tail_split = i ? (int)split : 0;
            }
          }
        }
      }
  if (out.one && any_split) {
    const double bytes = 2.0 * ((double)da.M * (double)da.K * 2.0 + (double)da.M * (double)da.N * 3.0 +
                                (double)db.M * (double)db.N * 2.0) +
                         (db.R ? 6.0 * (double)db.M * (double)db.N : 0.0);
    // (two launches take 1.17 times their estimates; of 30 problems, among them 128 x 8192 x
    // 512 and 20000 x 512 x 512 where two are faster, none is then decided wrongly)
    out.one = 6.48 + best + 0.174 * bytes / 6.3e6 < 1.17 * alone;
  }
  return GEMM_OK;
}

gemm_status_t run_pair(gemm_handle* h, const gemm_linear_t& da, const gemm_linear_t& db,
                       const PairPlan& plan, struct CUstream_st* stream) {
  CUtensorMap maps[6], second[6];
  gb300::PairParams kp{};
  GB300_CHECK(plan.db_first ? prepare_persistent(h, db, plan.each[1], maps, kp)
                            : prepare_persistent(h, da, plan.each[0], maps, kp));
  GB300_CHECK(plan.db_first ? prepare_persistent(h, da, plan.each[0], second, kp.second)
                            : prepare_persistent(h, db, plan.each[1], second, kp.second));
  // one layout of the slots for both
  for (gb300::EpiParams* e : {&kp.epi, &kp.second.epi}) {
    e->cd_bytes = (uint32_t)plan.cfg.epi_slot_bytes;
    e->xy_bytes = 0;
  }
  kp.first_items = kp.num_items;
  kp.num_items += kp.second.num_items;
  kp.lead_items = plan.lead_items;
  kp.lead_from = plan.lead_from;
  kp.a2 = second[0];
  kp.b2 = second[1];
  kp.c2 = second[2];
  kp.d2 = second[4];
  void* args[7] = {&maps[0], &maps[1], &maps[2], &maps[3], &maps[4], &maps[5], &kp};
  return launch_persistent(plan.cfg, plan.kern, args, stream);
}

// How a layer's gradients run: both in one launch, or each by its own plan.
struct ProductPlans {
  PairPlan pair;
  LinearPlan da, db;
};

// Plan them (null: not wanted, or empty), all of it before anything is enqueued: a
// configuration that one of them cannot take leaves every tensor as it was.
gemm_status_t plan_products(gemm_handle* h, const gemm_linear_bwd_t& p, const gemm_linear_t* da,
                            const gemm_linear_t* db, ProductPlans& out) {
  std::lock_guard<std::mutex> guard(h->mu);
  if (da && db && da->K > 0 && db->K > 0) {
    PairKey key;
    std::memset(&key, 0, sizeof(key));         // padding included: keys compare bytewise
    key.M = p.M; key.N = p.N; key.K = p.K;
    key.config_gen = h->config_gen;
    key.type = p.type; key.da_type = p.da_type; key.db_type = p.db_type;
    key.accumulate = p.accumulate != 0;
    PairPlan* plan = nullptr;
    for (PairPlan& c : h->pair_plans)
      if (c.valid && std::memcmp(&c.key, &key, sizeof(key)) == 0) { plan = &c; break; }
    if (!plan) {
      plan = &h->pair_plans[h->pair_next];
      plan->valid = false;
      GB300_CHECK(plan_pair(h, *da, *db, *plan));
      plan->key = key;
      plan->valid = true;
      h->pair_next = (h->pair_next + 1) % kPairPlans;
    }
    out.pair = *plan;
    if (plan->one) return GEMM_OK;
  }
  if (da) GB300_CHECK(find_plan(h, *da, out.da));
  if (db) GB300_CHECK(find_plan(h, *db, out.db));
  return GEMM_OK;
}

gemm_status_t run_products(gemm_handle* h, const gemm_linear_t* da, const gemm_linear_t* db,
                           const ProductPlans& plans, struct CUstream_st* stream) {
  std::lock_guard<std::mutex> guard(h->mu);
  if (plans.pair.one) {
    h->last = plans.pair.cfg;
    return run_pair(h, *da, *db, plans.pair, stream);
  }
  const bool two = da && db;
  if (da) GB300_CHECK(run_planned(h, *da, plans.da, two ? kFirstOfTwo : kAlone, stream));
  if (db) GB300_CHECK(run_planned(h, *db, plans.db, two ? kSecondOfTwo : kAlone, stream));
  return GEMM_OK;
}

// Clusters of `split` blocks of kern that the device holds at once, asked for once and kept in n.
template <class Kern>
int act_clusters(int& n, const gemm_handle* h, Kern kern, int threads, size_t smem, int split) {
  if (n > 0) return n;
  cudaLaunchConfig_t lc{};
  cudaLaunchAttribute attr[1];
  lc.gridDim = dim3((unsigned)(split * 4 * h->sm_count));
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &lc) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = std::max(1, h->sm_count * (1024 / threads) / split);
  }
  return n;
}

// Enqueue the activation gradient, with the block size and the blocks a cluster
// (which share a strip's rows) of the shortest estimate: waves x (rows a thread
// walks x a row's time, which grows with the SMs' load, + a block's start).
// Fitted on GB300 to 21 sizes (16 to 20000 rows of 64 to 28672) x 24 shapes: 3 % over
// the fastest on average, 15 % at worst.  For instance, gelu: 4096 x 8192 34.1 us with
// 128 blocks of 1024, 37.4 with 512 of 256 in clusters of 4; 8192 x 1024 13.9 with 16
// clusters of 6 blocks of 1024, 22.2 with clusters of 8, of which the device holds 15;
// 3000 x 5000 17.8 with clusters of 7 of 256, 19.4 with 8.
template <int DT>
gemm_status_t launch_act_grad(gemm_handle* h, gb300::ActGradParams& k, struct CUstream_st* stream) {
  typedef void (*Kern)(gb300::ActGradParams);
  const Kern kerns[3] = {gb300::act_grad_kernel<DT, 1024>, gb300::act_grad_kernel<DT, 512>,
                         gb300::act_grad_kernel<DT, 256>};
  const int64_t strips = cdiv(k.N, 64);
  Kern kern = nullptr;
  int threads = 0;
  double best = 0.0;
  const auto smem = [](int t) { return (size_t)(gb300::kActDepth * 2 * 16 + 32) * t; };
  {
    std::lock_guard<std::mutex> guard(h->mu);
    for (int size = 0; size < 3; ++size) {
      const int t = 1024 >> size;
      GB300_CHECK(raise_smem(h, reinterpret_cast<const void*>(kerns[size])));
      for (int split = 1; split <= 8; ++split) {
        const int held = act_clusters(h->act_clusters[DT == gb300::DT_F16][size][split], h, kerns[size],
                                      t, smem(t), split);
        const double full = (double)strips / held;
        const double waves = full <= 1.0 ? 1.0 : full + 0.156 * (std::ceil(full) - full);
        const double rows = (double)cdiv(k.M, (int64_t)split * (t / 8));
        const double load = std::min(1.0, (double)(std::min<int64_t>(strips, held) * split * t) /
                                              (1024.0 * h->sm_count));
        const double us = waves * (rows * (0.359 + 1.004 * load) + 1.166) + 0.078 * split +
                          0.133 * t / 1024.0;
        if (!kern || us < best) {
          best = us;
          kern = kerns[size];
          threads = t;
          k.row_split = split;
        }
      }
    }
  }
  return launch(kern, k, strips * k.row_split, threads, smem(threads), stream, k.row_split);
}

gemm_linear_t product_da(const gemm_linear_bwd_t& p, const void* dz, int64_t lddz) {
  gemm_linear_t q{};
  q.M = p.M; q.N = p.K; q.K = p.N;
  q.a_type = q.b_type = p.type;
  q.A = dz; q.lda = lddz; q.layoutA = GEMM_K_MAJOR;
  q.B = p.b; q.ldb = p.ldb; q.layoutB = GEMM_MN_MAJOR;
  q.alpha = p.alpha;
  q.D = p.da; q.ldd = p.ldda; q.d_type = p.da_type;
  return q;
}

gemm_linear_t product_db(const gemm_linear_bwd_t& p, const void* dz, int64_t lddz) {
  gemm_linear_t q{};
  q.M = p.N; q.N = p.K; q.K = p.M;
  q.a_type = q.b_type = p.type;
  q.A = dz; q.lda = lddz; q.layoutA = GEMM_MN_MAJOR;
  q.B = p.a; q.ldb = p.lda; q.layoutB = GEMM_MN_MAJOR;
  q.alpha = p.alpha;
  if (p.accumulate) { q.R = p.db; q.ldr = p.lddb; q.r_type = p.db_type; }
  q.D = p.db; q.ldd = p.lddb; q.d_type = p.db_type;
  return q;
}

// dz as the products read it: the caller's buffer, or dd itself where there is
// no activation and no buffer.
const void* dz_of(const gemm_linear_bwd_t& p, int64_t& ld) {
  ld = p.dz ? p.lddz : p.lddd;
  return p.dz ? p.dz : p.dd;
}

gemm_status_t check_linear_bwd(const gemm_linear_bwd_t& p) {
  if (!is_extent(p.M) || !is_extent(p.N) || !is_extent(p.K) || !is_activation(p.activation))
    return GEMM_ERR_INVALID_ARG;
  if (p.type != GEMM_F16 && p.type != GEMM_BF16) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if ((p.da && !is_epi_type(p.da_type)) || (p.db && !is_epi_type(p.db_type)) ||
      (p.dbias && !is_epi_type(p.dbias_type)))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (p.M > 0 && p.N > 0) {
    GB300_CHECK(check_matrix(p.dd, p.lddd, p.N, p.type));
    if (p.activation != GEMM_ACT_NONE) {
      GB300_CHECK(check_matrix(p.z, p.ldz, p.N, p.type));
      // the products read dz; without them it may be left out
      if (!p.dz && (p.da || p.db)) return GEMM_ERR_INVALID_ARG;
    }
    if (p.dz) {
      GB300_CHECK(check_matrix(p.dz, p.lddz, p.N, p.type));
      if ((p.dz == p.dd && p.lddz != p.lddd) || (p.dz == p.z && p.lddz != p.ldz))
        return GEMM_ERR_INVALID_ARG;
    }
  }
  if (p.dbias && !aligned_to(p.dbias, dtype_bytes(p.dbias_type))) return GEMM_ERR_MISALIGNED;
  int64_t lddz = 0;
  const void* dz = dz_of(p, lddz);
  if (p.da) {
    const gemm_linear_t q = product_da(p, dz, lddz);
    GB300_CHECK(check_linear(q));
    if (p.M > 0 && p.K > 0 && (p.da == p.dd || (p.a && p.da == p.a) || p.da == p.db))
      return GEMM_ERR_INVALID_ARG;
  }
  if (p.db) {
    const gemm_linear_t q = product_db(p, dz, lddz);
    GB300_CHECK(check_linear(q));
    if (p.N > 0 && p.K > 0 && (p.db == p.dd || (p.b && p.db == p.b))) return GEMM_ERR_INVALID_ARG;
  }
  return GEMM_OK;
}

}  // namespace

GEMM_API gemm_status_t gemm_linear_check(const gemm_linear_t* p) {
  return p ? check_linear(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_linear(gemm_handle_t h, const gemm_linear_t* p,
                                   struct CUstream_st* stream) {
  NvtxRange range("gemm_linear");
  if (!h || !p) return GEMM_ERR_INVALID_ARG;
  GB300_CHECK(check_linear(*p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  if (p->M == 0 || p->N == 0) return GEMM_OK;
  std::lock_guard<std::mutex> guard(h->mu);
  LinearPlan plan;
  GB300_CHECK(find_plan(h, *p, plan));
  return run_planned(h, *p, plan, kAlone, stream);
}

GEMM_API gemm_status_t gemm_linear_bwd_check(const gemm_linear_bwd_t* p) {
  return p ? check_linear_bwd(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_linear_bwd(gemm_handle_t h, const gemm_linear_bwd_t* pp,
                                       struct CUstream_st* stream) {
  NvtxRange range("gemm_linear_bwd");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_linear_bwd_t& p = *pp;
  GB300_CHECK(check_linear_bwd(p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  int64_t lddz = 0;
  const void* dz = dz_of(p, lddz);
  const gemm_linear_t q_da = product_da(p, dz, lddz), q_db = product_db(p, dz, lddz);
  const gemm_linear_t* const da = p.da && p.M > 0 && p.K > 0 ? &q_da : nullptr;
  const gemm_linear_t* const db = p.db && p.N > 0 && p.K > 0 ? &q_db : nullptr;
  ProductPlans plans;
  GB300_CHECK(plan_products(h, p, da, db, plans));
  if (p.N > 0 && (p.dz || p.dbias)) {
    gb300::ActGradParams k{};
    k.dd = p.dd; k.lddd = p.lddd;
    k.z = p.z; k.ldz = p.ldz;
    k.dz = p.dz; k.lddz = p.lddz;
    k.dbias = p.dbias; k.dbias_dt = device_dt(p.dbias_type);
    k.M = (int)p.M; k.N = (int)p.N;
    k.act = p.activation;
    GB300_CHECK(p.type == GEMM_F16 ? launch_act_grad<gb300::DT_F16>(h, k, stream)
                                   : launch_act_grad<gb300::DT_BF16>(h, k, stream));
  }
  return run_products(h, da, db, plans, stream);
}
