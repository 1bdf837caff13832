// The linear layer, D = act(alpha row_scale col_scale (A B^T) + bias) + R, and its
// backward pass (include/gemm_gb300.h): argument checks, planning and launches of
// the persistent kernel with the linear epilogue, and the activation-gradient
// kernel.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "activations.cuh"
#include "gemm_gb300.h"
#include "handle.h"
#include "kernels.h"
#include "rows.cuh"
#include "rows_host.h"

namespace gb300 {

struct ActGradParams {
  long long lddd, ldz, lddz;
  const void* dd;
  const void* z;                    // null: no activation, dz = dd
  void* dz;                         // or null: only the bias gradient is wanted
  void* dbias;                      // or null
  int M, N;
  int act, dbias_dt;
};

// dz = dd act'(z) and dbias = its column sums (of the values before dz is
// rounded).  A block owns 64 columns (8 lanes of one vector each) and walks all
// rows, 32 at a time; the 32 row groups' sums are added in order through shared
// memory.
template <int DT>
__global__ void __launch_bounds__(256)
act_grad_kernel(const __grid_constant__ ActGradParams p) {
  __shared__ float part[32][64];
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int es = elem_bytes(DT);
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int c = blockIdx.x * 64 + lane * kVec;
  float acc[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
  if (c < p.N) {
    with_activation(p.act, [&](auto a) {
      for (long long row = group; row < p.M; row += 32) {
        float g[kVec];
        load_vec<DT>(static_cast<const uint8_t*>(p.dd) + row * p.lddd * es, c, p.N, g);
        if constexpr (decltype(a)::value != ACT_NONE) {
          float z[kVec];
          load_vec<DT>(static_cast<const uint8_t*>(p.z) + row * p.ldz * es, c, p.N, z);
#pragma unroll
          for (int i = 0; i < kVec; ++i) g[i] *= activate_grad<decltype(a)::value>(z[i]);
        }
        if (p.dz) store_vec(static_cast<uint8_t*>(p.dz) + row * p.lddz * es, DT, c, p.N, g);
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[i] += g[i];
      }
    });
  }
  if (!p.dbias) return;
#pragma unroll
  for (int i = 0; i < kVec; ++i) part[group][lane * kVec + i] = acc[i];
  __syncthreads();
  const int col = blockIdx.x * 64 + (int)threadIdx.x;
  if (threadIdx.x < 64 && col < p.N) {
    float s = 0.f;
    for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
    store_elem(p.dbias, col, p.dbias_dt, s);
  }
}

}  // namespace gb300

namespace {

using namespace gb300host;

bool is_activation(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }

bool aligned_to(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

// Sizes the kernels index with 32 bits, and tensor-map strides below 2^40 bytes.
bool extent_ok(int64_t v) { return v >= 0 && v <= INT32_MAX; }
bool map_ok(int64_t ld, int64_t rows, int dt) {
  return (double)ld * dtype_bytes(dt) * (double)rows < 1099511627776.0;
}

// One A or B operand: `inner` contiguous elements a row, `rows` rows.
gemm_status_t check_operand(const void* p, int64_t ld, int64_t inner, int64_t rows, int dt) {
  GB300_CHECK(check_matrix(p, ld, inner, dt));
  return map_ok(ld, rows, dt) ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

gemm_status_t check_linear(const gemm_linear_t& p) {
  if (!extent_ok(p.M) || !extent_ok(p.N) || !extent_ok(p.K)) return GEMM_ERR_INVALID_ARG;
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

// Enqueue a checked call on the persistent kernel.
gemm_status_t run_persistent(gemm_handle* h, const gemm_linear_t& p, struct CUstream_st* stream) {
  const gemm_problem_t g = as_problem(p);
  std::lock_guard<std::mutex> guard(h->mu);
  gemm_config_t cfg{};
  GB300_CHECK(plan_valid(g, h->sm_count, h->smem_optin, h->forced ? &h->forced_cfg : nullptr, &cfg,
                         h->clusters_by_size, false,
                         EpilogueExtra{(int)gb300::kLinearSmem, activation_cost(p.activation)}));
  if (cfg.cluster_m != 1 || cfg.cluster_n != 1) return GEMM_ERR_UNSUPPORTED_CONFIG;
  const int es = dtype_bytes(p.a_type);
  const int ka = gb300::k_atoms(cfg.cta_group, cfg.tile_n);
  const void* kern = gb300::linear_kernel_for(es, cfg.cta_group, ka, cfg.epi_warps);
  if (!kern) return GEMM_ERR_UNSUPPORTED_CONFIG;
  VariantState& vs = h->linear_variants[es == 2 ? 0 : es == 1 ? 1 : 2][cfg.cta_group - 1][ka - 1]
                                       [cfg.epi_warps - 1];
  int resident = 0;
  GB300_CHECK(resident_kernel_clusters(h, vs, kern, cfg, cfg.cta_group, &resident));
  cfg.grid_ctas = (int)std::min<int64_t>(cfg.tiles + cfg.tail_split, resident) * cfg.cta_group;

  CUtensorMap maps[6];                 // A, B, C, X, D, Y
  std::memset(maps, 0, sizeof(maps));
  const bool a_mn = p.layoutA == GEMM_MN_MAJOR, b_mn = p.layoutB == GEMM_MN_MAJOR;
  if (p.K > 0 &&
      (!encode_operand(h->encode, &maps[0], p.A, p.a_type, p.M, p.K, 1, p.lda, a_mn, 128,
                       cfg.tile_k) ||
       !encode_operand(h->encode, &maps[1], p.B, p.b_type, p.N, p.K, 1, p.ldb, b_mn,
                       cfg.tile_n / cfg.cta_group, cfg.tile_k)))
    return GEMM_ERR_CUDA;
  if ((p.R && !encode_epi(h->encode, &maps[2], p.R, p.r_type, p.M, p.N, 1, false, p.ldr)) ||
      !encode_epi(h->encode, &maps[4], p.D, p.d_type, p.M, p.N, 1, false, p.ldd) ||
      (p.Z && !encode_epi(h->encode, &maps[5], p.Z, p.z_type, p.M, p.N, 1, false, p.ldz)))
    return GEMM_ERR_CUDA;

  KernelParams kp{};
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
  void* args[7] = {&maps[0], &maps[1], &maps[2], &maps[3], &maps[4], &maps[5], &kp};
  if (cudaLaunchKernelExC(&lc, kern, args) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  h->last = cfg;
  return GEMM_OK;
}

gemm_status_t run_linear(gemm_handle* h, const gemm_linear_t& p, struct CUstream_st* stream) {
  if (p.M == 0 || p.N == 0) return GEMM_OK;
  return run_persistent(h, p, stream);
}

// The backward pass's two products as linear calls.  da[M,K] = alpha dz[M,N] b[N,K]
// (b read N-major) and db[N,K] (+)= alpha dz^T a (both operands M-major).
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
  if (!extent_ok(p.M) || !extent_ok(p.N) || !extent_ok(p.K) || !is_activation(p.activation))
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
  return run_linear(h, *p, stream);
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
  if (p.N > 0 && (p.dz || p.dbias)) {
    gb300::ActGradParams k{};
    k.dd = p.dd; k.lddd = p.lddd;
    k.z = p.z; k.ldz = p.ldz;
    k.dz = p.dz; k.lddz = p.lddz;
    k.dbias = p.dbias; k.dbias_dt = device_dt(p.dbias_type);
    k.M = (int)p.M; k.N = (int)p.N;
    k.act = p.activation;
    GB300_CHECK(launch(p.type == GEMM_F16 ? gb300::act_grad_kernel<gb300::DT_F16>
                                          : gb300::act_grad_kernel<gb300::DT_BF16>,
                       k, cdiv(p.N, 64), 256, 0, stream));
  }
  int64_t lddz = 0;
  const void* dz = dz_of(p, lddz);
  if (p.da) GB300_CHECK(run_linear(h, product_da(p, dz, lddz), stream));
  if (p.db) GB300_CHECK(run_linear(h, product_db(p, dz, lddz), stream));
  return GEMM_OK;
}
