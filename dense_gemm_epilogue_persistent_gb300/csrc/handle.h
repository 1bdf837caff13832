// Host state shared by the library's entry-point units: the handle, its launch
// cache, NVTX ranges and the small helpers every argument check uses.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>
#include <mutex>

#include "gemm_gb300.h"
#include "gemm_kernel.cuh"

#define GEMM_API extern "C" __attribute__((visibility("default")))

namespace gb300host {

using gb300::KernelParams;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr uint64_t kDefaultTimeoutNs = 4000000000ull;
constexpr int kMaxStages = 12;
constexpr int kMaxEpiSlots = 6;

struct VariantState {
  bool smem_attr_set = false;  // max dynamic smem attribute raised to the opt-in limit
  int occ_smem = 0;            // dynamic smem size of the last occupancy query
  int max_clusters = 0;        // resident clusters at that size
};

// Everything a launch needs, prepared once per distinct call.  A call whose
// arguments (every field of the problem, byte for byte) and forced
// configuration equal a cached entry's launches from it without planning or
// encoding tensor maps again.
struct LaunchKey {
  gemm_problem_t problem;
  uint64_t config_gen;       // bumped by gemm_set_config
};

struct LaunchEntry {
  bool valid = false;
  LaunchKey key;
  gemm_config_t cfg{};
  const void* kern = nullptr;
  int cluster_ctas = 0;
  CUtensorMap maps[6];       // A, B, C, X, D, Y
  KernelParams kp{};
};

constexpr int kLaunchCacheEntries = 4;

// Plans of the linear layer's latest shapes.  A plan depends on sizes, layouts,
// types, activation and which tensors are there, never on an address.
struct SplitPlan {           // split-K kernel: tokens, features and CTAs of a tile, ring
  int bn, feats, split, ka, stages, smem;
  int64_t tiles_m, tiles_n;
};
struct LinearKey {
  int64_t M, N, K;
  uint64_t config_gen;
  int a_type, b_type, r_type, z_type, d_type, layoutA, layoutB, activation, has_r, has_z, plain;
};
struct LinearPlan {
  bool valid = false;
  LinearKey key;
  bool split = false;        // the split-K kernel, else the persistent one
  bool plain = false;        // ... the latter as the first of two products (is_plain)
  double us = 0.0;           // the estimate that it was chosen by
  SplitPlan s{};
  gemm_config_t cfg{};
  const void* kern = nullptr;
};
constexpr int kLinearPlans = 16;

// Plans of the latest two products run in one launch (the linear layer's
// gradients).
struct PairKey {
  int64_t M, N, K;
  uint64_t config_gen;
  int type, da_type, db_type, accumulate;
};
struct PairPlan {
  bool valid = false;
  PairKey key;
  bool one = false;          // one launch for both; else each by its own plan
  bool db_first = false;     // the items of db come first
  int lead_items = 0, lead_from = 0;   // as in PairParams
  gemm_config_t cfg{};       // tile, ring and grid
  gemm_config_t each[2]{};   // the same with each product's tiles (da, db)
  const void* kern = nullptr;
};
constexpr int kPairPlans = 8;

// NVTX ranges in the "gemm_gb300" domain around every entry point that
// enqueues work (and around planning and tensor-map encoding on a launch-cache
// miss), so that a profiler's timeline and its range filters (ncu --nvtx
// --nvtx-include "gemm_gb300@gemm_run/") can pick the library's calls out.
// Without a tool attached each push and pop returns at once.
inline nvtxDomainHandle_t nvtx_domain() {
  static const nvtxDomainHandle_t d = nvtxDomainCreateA("gemm_gb300");
  return d;
}

struct NvtxRange {
  explicit NvtxRange(const char* name) {
    nvtxEventAttributes_t a{};
    a.version = NVTX_VERSION;
    a.size = NVTX_EVENT_ATTRIB_STRUCT_SIZE;
    a.messageType = NVTX_MESSAGE_TYPE_ASCII;
    a.message.ascii = name;
    nvtxDomainRangePushEx(nvtx_domain(), &a);
  }
  ~NvtxRange() { nvtxDomainRangePop(nvtx_domain()); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace gb300host

struct gemm_handle {
  int device = 0;
  int sm_count = 0;
  int smem_optin = 0;
  gb300host::EncodeTiledFn encode = nullptr;
  uint32_t* d_status = nullptr;
  bool forced = false;
  gemm_config_t forced_cfg{};
  gemm_config_t last{};
  bool counted = true;         // the latest launch is of a kernel with ring counters
  uint64_t timeout_ns = gb300host::kDefaultTimeoutNs;
  gb300host::VariantState variants[3][2][2][2][2][2][2];   // [ab 16/8/32][cta_group][k atoms][mc][nc][epw][sk]
  gb300host::VariantState linear_variants[3][2][2][2];   // [ab][cta_group][k atoms][epw]
  gb300host::VariantState pair_variants[2][2][2];        // [cta_group][k atoms][epw]
  int clusters_by_size[9] = {0, 0, 0, 0, 0, 0, 0, 0, 0};   // resident clusters of 1, 2, 4, 8 CTAs
  uint64_t config_gen = 0;
  gb300host::LaunchEntry cache[gb300host::kLaunchCacheEntries];
  int cache_next = 0;
  gb300host::LinearPlan linear_plans[gb300host::kLinearPlans];
  int linear_next = 0;
  gb300host::PairPlan pair_plans[gb300host::kPairPlans];
  int pair_next = 0;
  gb300host::VariantState grouped_variants[3][2][3][4];  // [ab][cta_group][form][lean epilogue's type + 1]
  int route_cluster = 0;      // blocks of the sort's cluster (0: not asked)
  int split_clusters[9] = {0, 0, 0, 0, 0, 0, 0, 0, 0};   // resident, by cluster size (0: not asked)
  int act_clusters[3][2][3][9] = {};   // activation gradient's, by form, type, block size and cluster
  std::mutex mu;
  void* ws = nullptr;          // gemm_run_host's device copies of its host buffers
  size_t ws_bytes = 0;
  std::mutex ws_mu;
  unsigned long long* d_stats = nullptr;   // ring statistics (statistics build only)
  // Kernels whose dynamic shared-memory limit this handle has raised.
  static constexpr int kMaxRaised = 64;
  const void* raised[kMaxRaised] = {};
  int raised_count = 0;
  // Stream-K workspace: one 128 x 256 fp32 partial slot and one flag per SM
  // (null: stream-K is never planned for this handle).
  float* sk_partials = nullptr;
  uint32_t* sk_flags = nullptr;
};

namespace gb300host {

inline int dtype_bytes(int dt) {
  switch (dt) {
    case GEMM_F32: return 4;
    case GEMM_F16: return 2;
    case GEMM_BF16: return 2;
    case GEMM_E4M3: return 1;
    case GEMM_E5M2: return 1;
    case GEMM_TF32: return 4;
  }
  return 0;
}

inline bool is_epi_type(int dt) { return dt == GEMM_F32 || dt == GEMM_F16 || dt == GEMM_BF16; }
inline bool is_fp8(int dt) { return dt == GEMM_E4M3 || dt == GEMM_E5M2; }
inline bool is_ab_type(int dt) {
  return dt == GEMM_F16 || dt == GEMM_BF16 || is_fp8(dt) || dt == GEMM_TF32;
}
inline bool is_layout(int v) { return v == GEMM_K_MAJOR || v == GEMM_MN_MAJOR; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// B's type: the descriptor's b when set (0 = GEMM_F32 means "same as ab").
inline int b_type(const gemm_dtypes_t& t) { return t.b == GEMM_F32 ? t.ab : t.b; }

inline bool reads_c(const gemm_problem_t& p) { return p.beta != 0.0f; }
inline bool reads_x(const gemm_problem_t& p) { return p.X != nullptr && p.x_factor != 0.0f; }

// What the linear layer's epilogue adds to a plan: its own cost model, shared
// memory per CTA, and the activation's time per 32-column chunk.
struct EpilogueExtra {
  bool linear = false;
  int smem = 0;
  double chunk_cost = 0.0;
};

// gemm_api.cu: the planner on a problem whose arguments have been checked, and
// what a launch is prepared with (described at their definitions).
gemm_status_t plan_valid(const gemm_problem_t& p, int sm_count, int smem_optin,
                         const gemm_config_t* forced, gemm_config_t* out,
                         const int* clusters_by_size, bool stream_k_ok,
                         const EpilogueExtra& extra, double* cost = nullptr);
bool encode_operand(EncodeTiledFn enc, CUtensorMap* map, const void* ptr, int dt, int64_t rows,
                    int64_t K, int64_t L, int64_t ld, bool mn_major, int box_rows, int tile_k);
bool encode_stack(EncodeTiledFn enc, CUtensorMap* map, const void* ptr, int dt, int64_t inner,
                  int64_t rows, int64_t sets, int64_t ld, int64_t stride, int box_rows);
bool encode_epi(EncodeTiledFn enc, CUtensorMap* map, const void* ptr, int dt, int64_t M,
                int64_t N, int64_t L, bool m_major, int64_t ld);
uint32_t make_idesc(int a_type, int b_type_, bool acc_f16, int cg, int bn, bool a_mn, bool b_mn);
gemm_status_t resident_kernel_clusters(const gemm_handle* h, VariantState& vs, const void* kern,
                                       const gemm_config_t& cfg, int csize, int* clusters);

// Whether the calling thread's current device is the handle's.
inline bool on_device(const gemm_handle* h) {
  int cur = -1;
  if (cudaGetDevice(&cur) == cudaSuccess && cur == h->device) return true;
  cudaGetLastError();
  return false;
}

}  // namespace gb300host
