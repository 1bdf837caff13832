// The linear layer over groups of rows with weights of their own, its backward pass, and
// low-rank adapters (include/gemm_gb300.h): argument checks, planning and launches of
// the kernel in grouped_kernel.cuh.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "adapters_few.cuh"
#include "gemm_gb300.h"
#include "grouped_kernel.cuh"
#include "handle.h"
#include "kernels.h"
#include "rows_host.h"

namespace {

using namespace gb300host;

// One launch of the kernel.  Rows form: F the weights [sets][feats, k] (f_mn: [k, feats]),
// T the tokens [rows, k].  Weights form: F the tokens' inputs [rows, feats], T the
// gradients of their outputs [rows, cols].
struct Product {
  bool weights = false;
  int64_t rows = 0, feats = 0, cols = 0, k = 0, groups = 0, sets = 0;
  gemm_dtype_t f_type{}, t_type{};
  bool f_mn = false;
  const void* f = nullptr; int64_t ldf = 0, stride_f = 0;
  const void* t = nullptr; int64_t ldt = 0;
  gb300::GroupedParams k_params{};     // the epilogue's part, offsets and index
};

// The type of the lean epilogue, or -1 for the whole one: nothing but alpha, a set's scale and a
// residual of d's type; the 16-bit forms move features, and read a residual's, by twos.  (8191 x 8192 of inner size 64 with
// a residual, bf16: 66 us, 125 by the whole one.)
int lean_of(const Product& p) {
  const gb300::GroupedParams& k = p.k_params;
  const int dt = device_dt(k.d_dt);
  const bool lean = dtype_bytes(p.f_type) == 2 && !k.row_scale && !k.col_scale && !k.bias && !k.z &&
                    k.act == gb300::ACT_NONE && (!k.r || k.r_dt == k.d_dt) &&
                    (dt == gb300::DT_F32 || p.feats % 2 == 0 || !k.r);
  return lean ? dt : -1;
}

struct GroupedPlan {
  gemm_config_t cfg{};
  int form = gb300::kGroupedRows, lean = -1;
  const void* kern = nullptr;
};

// Columns of the token operand's boxes: a tile's width is a multiple of this x cta_group.
int box_unit(bool weights, int cta_group, int bn) {
  return weights ? 64 : cta_group == 2 ? 32 : bn % 32 == 0 && bn > 64 ? 32 : 16;
}

// Features of a ring stage: a single narrow tile's own leave room for more stages.  (Adapters' first
// product, 8191 rows of 4096 by 7 x 64 bf16: 24.1 us with 128, 21.5 so.)
int f_rows_of(const Product& p) {
  return !p.weights && !p.f_mn && p.feats < 128 ? (int)cdiv(p.feats, 8) * 8 : 128;
}

// Feature tiles x column tiles: the items of a launch, at most (the device finds out how
// many there are).
int64_t items_of(const Product& p, const gemm_config_t& c) {
  const int64_t tiles_f = cdiv(p.feats, c.tile_m);
  return p.weights ? p.groups * tiles_f * cdiv(p.cols, c.tile_n)
                   : (p.rows / c.tile_n + std::min(p.groups, p.rows)) * tiles_f;
}

// An estimate, microseconds, of the rows form with tiles of `bn` tokens: the launch and a first item's
// k-blocks and epilogue, then rounds of items at the pace of their loads or their epilogues.  Fitted on
// GB300 to 40 to 9600 rows in 1 to 32 uneven groups, 512 to 4096 features of inner sizes 512 and 2048 bf16,
// with gelu and without: over those the choice is 1 % slower than the best of its three tiles (1.5 % than the best of
// five, single CTAs with 128 and 256 among them), 10 % (gelu) and 5 %
// faster than the widest wherever groups have more than 64 rows.  (600 rows of 8 groups, 1024 x 512: 7.4 us with
// single tiles, 9.0 with the widest; 300 of one, 2048 x 512 6.8, 12.3; 2400 of 8, 512 x 2048 13.5 with pairs of 128, 18.9.)
double rows_us(const gemm_handle* h, const Product& p, int cg, int bn, bool lean) {
  const double groups = (double)std::max<int64_t>(1, std::min(p.groups, p.rows));
  const double mean = (double)p.rows / groups, width = std::min((double)bn, mean);
  const double tiles = groups > 1 ? groups * (mean > 0.5 * bn ? std::max(1.0, mean / bn + 0.5) : 1.0)
                                  : (double)cdiv(p.rows, bn);
  const double items = tiles * (double)cdiv(p.feats, 128 * cg);
  const double rounds = std::max(1.0, std::ceil(items / (h->sm_count / cg)));
  const double blocks = (double)cdiv(p.k * dtype_bytes(p.f_type), 128 * gb300::kGroupedKA);
  const double first = cg == 1 ? 0.35 : bn == 128 ? 0.30 : 0.45;
  const double block = cg == 1 ? 0.41 : 0.22 + 0.0018 * width;
  const double whole = lean ? (cg == 1 ? 1.8 : bn == 128 ? 2.6 : 4.0) : (cg == 1 ? 2.4 : bn == 128 ? 3.9 : 7.3);
  const double epilogue = whole * std::max(0.25, width / bn);
  return 4.2 + first * blocks + epilogue + (rounds - 1) * std::max(block * blocks, epilogue);
}

// A launch's tile.
gemm_status_t choose_tile(const gemm_handle* h, const Product& p, gemm_config_t& c) {
  const gemm_config_t f = h->forced ? h->forced_cfg : gemm_config_t{};
  if (f.cluster_m > 1 || f.cluster_n > 1 || f.split_k > 0 || f.stream_k > 1)
    return GEMM_ERR_UNSUPPORTED_CONFIG;
  const int64_t mean = cdiv(p.rows, std::max<int64_t>(1, std::min(p.groups, p.rows)));
  if (p.weights)
    c.cta_group = p.groups * cdiv(p.feats, 256) * cdiv(p.cols, 256) * 2 > h->sm_count / 2 ? 2 : 1;
  else
    c.cta_group = p.feats > 128 && mean > 64 ? 2 : 1;
  if (f.cta_group) c.cta_group = f.cta_group;
  // (of very short groups narrow tiles, which leave room for more stages: 2 rows of 8 experts, 2048 x 8192 27.0 us with
  // 16, 31.2 with 64; 8 of 16, 512 x 4096 16.0, 18.1; 400 of 32, 1024 x 2048 25.4 with 32, 29.2 with 16, 26.2 with 64)
  c.tile_n = c.cta_group == 2 ? 256 : p.weights ? 128 : f.cta_group ? 64 : mean <= 4 ? 16 : mean <= 16 ? 32 : 64;
  if (!p.weights && c.cta_group == 2 && !f.cta_group && !f.tile_n) {
    const bool lean = lean_of(p) >= 0;
    const double widest = rows_us(h, p, 2, 256, lean), pairs = rows_us(h, p, 2, 128, lean),
                 single = rows_us(h, p, 1, 64, lean);
    if (single < widest && single < pairs) { c.cta_group = 1; c.tile_n = 64; }
    else if (pairs < widest) c.tile_n = 128;
  }
  if (f.tile_n) c.tile_n = f.tile_n;
  c.tile_m = 128 * c.cta_group;
  return c.tile_n % (box_unit(p.weights, c.cta_group, c.tile_n) * c.cta_group) == 0
             ? GEMM_OK : GEMM_ERR_UNSUPPORTED_CONFIG;
}

// The rest of a plan whose tile, form and epilogue are chosen (h->mu held).  `items`: at most so many.
gemm_status_t finish_plan(gemm_handle* h, const Product& p, int64_t items, GroupedPlan& out) {
  const int es = dtype_bytes(p.f_type), f_rows = f_rows_of(p);
  const gemm_config_t f = h->forced ? h->forced_cfg : gemm_config_t{};
  gemm_config_t& c = out.cfg;
  const auto smem = [&](int stages) {
    return gb300::grouped_smem(c.cta_group, c.tile_n, f_rows, stages, (int)p.groups);
  };
  c.stages = 0;
  while (c.stages < gb300::kGroupedMaxStages && smem(c.stages + 1) <= h->smem_optin) ++c.stages;
  if (f.stages) {
    if (f.stages > c.stages) return GEMM_ERR_UNSUPPORTED_CONFIG;
    c.stages = f.stages;
  }
  if (c.stages < 1) return GEMM_ERR_UNSUPPORTED_CONFIG;
  // (more than half an SM's shared memory: one CTA an SM, which owns its tensor memory)
  c.smem_bytes = std::max(smem(c.stages), h->smem_optin / 2 + 1024);
  c.tile_k = 128 / es * gb300::kGroupedKA;
  c.acc_stages = gb300::kAccStages;
  c.ring_bytes = c.stages * gb300::grouped_stage_bytes(c.cta_group, c.tile_n, f_rows);
  c.cluster_m = c.cluster_n = 1;
  c.epi_warps = gb300::grouped_streams(out.lean);
  c.inject_stall = f.inject_stall;
  c.group_m = f.group_m ? std::min(f.group_m, gb300::kGroupedMaxStrip) : 8;
  c.tiles = items;
  if (c.tiles > INT32_MAX / 2) return GEMM_ERR_INVALID_ARG;
  out.kern = gb300::grouped_kernel_for(es, c.cta_group, out.form, out.lean);
  if (!out.kern) return GEMM_ERR_UNSUPPORTED_CONFIG;
  int resident = 0;
  gemm_config_t asked = c;
  asked.epi_warps = 2;                 // (the threads that resident_kernel_clusters counts: one CTA an SM anyway)
  GB300_CHECK(resident_kernel_clusters(
      h, h->grouped_variants[es == 2 ? 0 : es == 1 ? 1 : 2][c.cta_group - 1][out.form][out.lean + 1],
      out.kern, asked, c.cta_group, &resident));
  c.grid_ctas = (int)std::max<int64_t>(1, std::min<int64_t>(c.tiles, resident)) * c.cta_group;
  return GEMM_OK;
}

// Plan one product (h->mu held).
gemm_status_t plan_grouped(gemm_handle* h, const Product& p, GroupedPlan& out) {
  GB300_CHECK(choose_tile(h, p, out.cfg));
  out.form = p.weights ? gb300::kGroupedWeights : gb300::kGroupedRows;
  out.lean = lean_of(p);
  return finish_plan(h, p, items_of(p, out.cfg), out);
}

// Plan both gradients as one launch, where one lean epilogue suits both (h->mu held); out.kern stays null
// where not.  The tile is the weight gradient's, or pairs of 128 where that alone would take single
// ones: what a launch of their own would gain by other tiles is less than it costs.  (One launch, two with
// tiles of their own: 100 rows of one group, 512 x 512 7.4 us, 11.0; of 6, 1024 x 1024 12.3, 16.4; 2400 of one, 1024 x
// 1024 17.1, 21.5; 2002 of 6, 2003 x 1501 38.2, 42.3; 8192 of 16, 4096 x 4096 452, 466; the other way round where many
// groups have few rows of large weights: 100 of 64, 2048 x 2048 197, 189.)
gemm_status_t plan_both(gemm_handle* h, const Product& da, const Product& db, GroupedPlan& out) {
  gemm_config_t ca{};
  GB300_CHECK(choose_tile(h, da, ca));
  GB300_CHECK(choose_tile(h, db, out.cfg));
  out.lean = lean_of(da);
  if (out.lean < 0 || lean_of(db) != out.lean) return GEMM_OK;
  if (h->forced || da.feats <= 128) {
    if (ca.cta_group != out.cfg.cta_group || ca.tile_n != out.cfg.tile_n) return GEMM_OK;
  } else if (out.cfg.cta_group == 1) {
    out.cfg.cta_group = 2;
    out.cfg.tile_n = 128;
    out.cfg.tile_m = 256;
  }
  out.form = gb300::kGroupedBoth;
  return finish_plan(h, da, items_of(da, out.cfg) + items_of(db, out.cfg), out);
}

// A product's tensor maps (`whole`: a whole tile's tokens, of the rows form) and parameters by its plan.
gemm_status_t prepare(gemm_handle* h, const Product& p, const gemm_config_t& c, CUtensorMap& f,
                      CUtensorMap& t, CUtensorMap* whole, gb300::GroupedParams& k) {
  const int unit = box_unit(p.weights, c.cta_group, c.tile_n);
  std::memset(&f, 0, sizeof(f));
  std::memset(&t, 0, sizeof(t));
  if (whole) std::memset(whole, 0, sizeof(*whole));
  k = p.k_params;
  k.has_operands = p.weights ? p.rows > 0 : p.k > 0;
  if (k.has_operands) {
    const int box = gb300::kGroupedMBox;
    const int64_t sets = p.stride_f ? p.sets : 1;      // (a map's stride may not be 0)
    const bool ok =
        p.weights
            ? encode_stack(h->encode, &f, p.f, p.f_type, p.feats, p.rows, 1, p.ldf, 0, box) &&
                  encode_stack(h->encode, &t, p.t, p.t_type, p.cols, p.rows, 1, p.ldt, 0, box)
            : (p.f_mn ? encode_stack(h->encode, &f, p.f, p.f_type, p.feats, p.k, sets, p.ldf,
                                     p.stride_f, c.tile_k)
                      : encode_stack(h->encode, &f, p.f, p.f_type, p.k, p.feats, sets, p.ldf,
                                     p.stride_f, f_rows_of(p))) &&
                  encode_stack(h->encode, &t, p.t, p.t_type, p.k, p.rows, 1, p.ldt, 0, unit) &&
                  encode_stack(h->encode, whole, p.t, p.t_type, p.k, p.rows, 1, p.ldt, 0,
                               c.tile_n / c.cta_group);
    if (!ok) return GEMM_ERR_CUDA;
  }
  k.rows = (int)p.rows; k.feats = (int)p.feats; k.cols = (int)p.cols; k.k = (int)p.k;
  k.groups = (int)p.groups; k.sets = (int)p.sets;
  k.bn = c.tile_n;
  k.unit = unit;
  k.f_rows = f_rows_of(p);
  k.tiles_f = (int)cdiv(p.feats, c.tile_m);
  k.tiles_c = p.weights ? (int)cdiv(p.cols, c.tile_n) : 1;
  k.stages = c.stages;
  k.strip = c.group_m;
  k.set_step = p.stride_f != 0;
  k.by_bn = gb300::fast_div(k.bn);
  k.by_strip = gb300::fast_div(k.strip * k.tiles_f);
  k.by_group = gb300::fast_div(k.tiles_f * k.tiles_c);
  k.alternate = 1;
  k.f_mn = p.f_mn;
  k.idesc = make_idesc(p.f_type, p.t_type, false, c.cta_group, 0, p.weights || p.f_mn, p.weights);
  k.status = h->d_status;
  k.timeout_ns = h->timeout_ns;
  k.inject_stall = c.inject_stall;
  return GEMM_OK;
}

// Enqueue a planned launch (h->mu held); args: its tensor maps and parameters.
gemm_status_t launch_planned(gemm_handle* h, const GroupedPlan& plan, void** args,
                             struct CUstream_st* stream) {
  const gemm_config_t& c = plan.cfg;
  cudaLaunchConfig_t lc{};
  cudaLaunchAttribute attr[2];
  lc.gridDim = dim3((unsigned)c.grid_ctas);
  lc.blockDim = dim3((unsigned)gb300::grouped_threads(plan.form, plan.lean));
  lc.dynamicSmemBytes = (size_t)c.smem_bytes;
  lc.stream = reinterpret_cast<cudaStream_t>(stream);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)c.cta_group;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = c.cta_group > 1 ? 2 : 1;
  h->last = c;
  h->counted = false;
  if (cudaLaunchKernelExC(&lc, plan.kern, args) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

gemm_status_t run_grouped(gemm_handle* h, const Product& p, const GroupedPlan& plan,
                          struct CUstream_st* stream) {
  CUtensorMap f, t, whole;
  gb300::GroupedParams k{};
  GB300_CHECK(prepare(h, p, plan.cfg, f, t, &whole, k));
  void* args[4] = {&f, &t, &whole, &k};
  return launch_planned(h, plan, args, stream);
}

gemm_status_t run_both(gemm_handle* h, const Product& da, const Product& db, const GroupedPlan& plan,
                       struct CUstream_st* stream) {
  CUtensorMap f, t, whole;
  gb300::GroupedBothParams k{};
  GB300_CHECK(prepare(h, da, plan.cfg, f, t, &whole, k));
  GB300_CHECK(prepare(h, db, plan.cfg, k.f2, k.t2, nullptr, k.weights));
  void* args[4] = {&f, &t, &whole, &k};
  return launch_planned(h, plan, args, stream);
}

bool is_count(int64_t v) { return v >= 0 && v <= gb300::kGroupedMaxGroups; }

// Offsets, and an index where there is one.
gemm_status_t check_groups(const int32_t* offsets, const int32_t* index) {
  if (!offsets) return GEMM_ERR_INVALID_ARG;
  return aligned_to(offsets, 4) && aligned_to(index, 4) ? GEMM_OK : GEMM_ERR_MISALIGNED;
}

// `sets` matrices of `rows` rows of `inner` contiguous elements, `stride` apart.
gemm_status_t check_stack(const void* p, int64_t ld, int64_t inner, int64_t rows, int64_t sets,
                          int64_t stride, int dt) {
  GB300_CHECK(check_operand(p, ld, inner, rows, dt));
  if (sets <= 1) return GEMM_OK;
  if (stride < 0 || (stride * dtype_bytes(dt)) % 16 != 0) return GEMM_ERR_MISALIGNED;
  return map_ok(stride, 1, dt) ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

// Matrices that are written may not lie on one another.
bool apart(int64_t stride, int64_t ld, int64_t rows, int64_t cols, int64_t sets) {
  return sets <= 1 || rows == 0 || stride >= (rows - 1) * ld + cols;
}

// Feature tiles x token tiles of any grouping fit the items' numbers.
bool items_ok(int64_t rows, int64_t groups, int64_t feats) {
  return (cdiv(rows, 16) + groups) * cdiv(feats, 128) <= INT32_MAX / 2;
}

gemm_status_t check_grouped(const gemm_grouped_linear_t& p) {
  if (!is_extent(p.M) || !is_extent(p.N) || !is_extent(p.K) || !is_count(p.groups) ||
      !is_count(p.sets) || (!p.index && p.sets < p.groups))
    return GEMM_ERR_INVALID_ARG;
  if (!is_layout(p.layoutB) || !is_activation(p.activation)) return GEMM_ERR_INVALID_ARG;
  if (!is_ab_type(p.a_type) || !is_ab_type(p.b_type) ||
      (p.a_type != p.b_type && !(is_fp8(p.a_type) && is_fp8(p.b_type))))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (p.a_type == GEMM_TF32 && p.layoutB != GEMM_K_MAJOR) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (!is_epi_type(p.d_type) || (p.bias && !is_epi_type(p.bias_type)) ||
      (p.R && !is_epi_type(p.r_type)) || (p.Z && !is_epi_type(p.z_type)))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (p.M == 0 || p.N == 0 || p.groups == 0) return GEMM_OK;
  GB300_CHECK(check_groups(p.offsets, p.index));
  if (!items_ok(p.M, p.groups, p.N)) return GEMM_ERR_INVALID_ARG;
  GB300_CHECK(check_operand(p.D, p.ldd, p.N, p.M, p.d_type));
  if (p.R) GB300_CHECK(check_operand(p.R, p.ldr, p.N, p.M, p.r_type));
  if (p.Z) GB300_CHECK(check_operand(p.Z, p.ldz, p.N, p.M, p.z_type));
  if (p.K > 0 && p.sets > 0) {
    const bool bn = p.layoutB == GEMM_MN_MAJOR;
    GB300_CHECK(check_operand(p.A, p.lda, p.K, p.M, p.a_type));
    GB300_CHECK(check_stack(p.B, p.ldb, bn ? p.N : p.K, bn ? p.K : p.N, p.sets, p.strideB, p.b_type));
  }
  if (!aligned_to(p.row_scale, 4) || !aligned_to(p.col_scale, 4) ||
      (p.bias && !aligned_to(p.bias, dtype_bytes(p.bias_type))))
    return GEMM_ERR_MISALIGNED;
  // in place: element for element only; nothing else may share an output
  if (p.R == p.D && (p.r_type != p.d_type || p.ldr != p.ldd)) return GEMM_ERR_INVALID_ARG;
  for (const void* out : {(const void*)p.D, (const void*)p.Z})
    if (same_place(out, {p.offsets, p.index, p.row_scale, p.col_scale, p.bias}) ||
        (p.K > 0 && same_place(out, {p.A, p.B})))
      return GEMM_ERR_INVALID_ARG;
  if (same_place(p.Z, {p.D, p.R})) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

Product product_of(const gemm_grouped_linear_t& p) {
  Product q;
  q.rows = p.M; q.feats = p.N; q.groups = p.groups; q.sets = p.sets;
  q.k = p.sets > 0 ? p.K : 0;          // (no group has weights)
  q.f_type = p.b_type; q.t_type = p.a_type;
  q.f_mn = p.layoutB == GEMM_MN_MAJOR;
  q.f = p.B; q.ldf = p.ldb; q.stride_f = p.strideB;
  q.t = p.A; q.ldt = p.lda;
  gb300::GroupedParams& k = q.k_params;
  k.offsets = p.offsets; k.index = p.index;
  k.alpha = p.alpha;
  k.row_scale = p.row_scale; k.col_scale = p.col_scale;
  k.bias = p.bias; k.bias_dt = p.bias_type;
  k.r = p.R; k.ldr = p.ldr; k.r_dt = p.r_type;
  k.z = p.Z; k.ldz = p.ldz; k.z_dt = p.z_type;
  k.d = p.D; k.ldd = p.ldd; k.d_dt = p.d_type;
  k.act = p.activation;
  k.skip_none = p.R == p.D && !p.Z;
  return q;
}

// dz as the products read it: the caller's buffer, or dd itself where there is no
// activation and no buffer.
const void* dz_of(const gemm_grouped_linear_bwd_t& p, int64_t& ld) {
  ld = p.dz ? p.lddz : p.lddd;
  return p.dz ? p.dz : p.dd;
}

Product product_da(const gemm_grouped_linear_bwd_t& p, const void* dz, int64_t lddz) {
  Product q;
  q.rows = p.M; q.feats = p.K; q.k = p.N; q.groups = q.sets = p.groups;
  q.f_type = q.t_type = p.type;
  q.f_mn = true;
  q.f = p.b; q.ldf = p.ldb; q.stride_f = p.strideb;
  q.t = dz; q.ldt = lddz;
  gb300::GroupedParams& k = q.k_params;
  k.offsets = p.offsets;
  k.alpha = p.alpha;
  k.d = p.da; k.ldd = p.ldda; k.d_dt = p.da_type;
  return q;
}

Product product_db(const gemm_grouped_linear_bwd_t& p, const void* dz, int64_t lddz) {
  Product q;
  q.weights = true;
  q.rows = p.M; q.feats = p.K; q.cols = p.N; q.groups = q.sets = p.groups;
  q.f_type = q.t_type = p.type;
  q.f = p.a; q.ldf = p.lda;
  q.t = dz; q.ldt = lddz;
  gb300::GroupedParams& k = q.k_params;
  k.offsets = p.offsets;
  k.alpha = p.alpha;
  k.d = p.db; k.ldd = p.lddb; k.sd = p.stridedb; k.d_dt = p.db_type;
  if (p.accumulate) { k.r = p.db; k.ldr = p.lddb; k.r_dt = p.db_type; }
  return q;
}

// Without features there is nothing to compute but da, the sum of nothing, in the groups' rows.
bool no_gradient(const gemm_grouped_linear_bwd_t& p) {
  return p.groups == 0 || (p.N == 0 && (!p.da || p.M == 0 || p.K == 0 || !p.offsets));
}

gemm_status_t check_grouped_bwd(const gemm_grouped_linear_bwd_t& p) {
  if (!is_extent(p.M) || !is_extent(p.N) || !is_extent(p.K) || !is_count(p.groups) ||
      !is_activation(p.activation))
    return GEMM_ERR_INVALID_ARG;
  if (p.type != GEMM_F16 && p.type != GEMM_BF16) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if ((p.da && !is_epi_type(p.da_type)) || (p.db && !is_epi_type(p.db_type)) ||
      (p.dbias && !is_epi_type(p.dbias_type)))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (no_gradient(p)) return GEMM_OK;
  GB300_CHECK(check_groups(p.offsets, nullptr));
  if (cdiv(p.N, 64) * p.groups > INT32_MAX / 8 || !items_ok(p.M, p.groups, p.K) ||
      p.groups * cdiv(p.K, 128) * cdiv(p.N, 64) > INT32_MAX / 2)
    return GEMM_ERR_INVALID_ARG;
  if (p.N == 0) return check_operand(p.da, p.ldda, p.K, p.M, p.da_type);
  if (p.M > 0) {
    GB300_CHECK(check_operand(p.dd, p.lddd, p.N, p.M, p.type));
    if (p.activation != GEMM_ACT_NONE) {
      GB300_CHECK(check_operand(p.z, p.ldz, p.N, p.M, p.type));
      // the products read dz; without them it may be left out
      if (!p.dz && (p.da || p.db)) return GEMM_ERR_INVALID_ARG;
    }
    if (p.dz) {
      GB300_CHECK(check_operand(p.dz, p.lddz, p.N, p.M, p.type));
      if ((p.dz == p.dd && p.lddz != p.lddd) || (p.dz == p.z && p.lddz != p.ldz))
        return GEMM_ERR_INVALID_ARG;
    }
  }
  if (p.dbias && !aligned_to(p.dbias, dtype_bytes(p.dbias_type))) return GEMM_ERR_MISALIGNED;
  // no output where another tensor of the call lies that is read or written: dz is complete before a and b
  // are read, dbias before dz is
  const void* const da = p.M > 0 && p.K > 0 ? p.da : nullptr;
  const void* const db = p.K > 0 ? p.db : nullptr;
  const void* const a = db && p.M > 0 ? p.a : nullptr;
  const void* const b = da ? p.b : nullptr;
  if (same_place(p.dbias, {p.offsets, a, b, da, db}) || same_place(da, {p.offsets}) ||
      same_place(db, {p.offsets}))
    return GEMM_ERR_INVALID_ARG;
  if (p.M > 0 && (same_place(p.dz, {p.offsets, a, b, p.dbias, da, db}) || same_place(p.dbias, {p.dd, p.z})))
    return GEMM_ERR_INVALID_ARG;
  if (p.K == 0) return GEMM_OK;
  int64_t lddz = 0;
  const void* dz = dz_of(p, lddz);
  if (p.da && p.M > 0) {
    GB300_CHECK(check_operand(p.da, p.ldda, p.K, p.M, p.da_type));
    GB300_CHECK(check_stack(p.b, p.ldb, p.K, p.N, p.groups, p.strideb, p.type));
    if (p.da == p.dd || p.da == dz || p.da == p.z || p.da == p.a || p.da == p.b || p.da == p.db)
      return GEMM_ERR_INVALID_ARG;
  }
  if (p.db) {
    GB300_CHECK(check_stack(p.db, p.lddb, p.K, p.N, p.groups, p.stridedb, p.db_type));
    if (!apart(p.stridedb, p.lddb, p.N, p.K, p.groups)) return GEMM_ERR_INVALID_ARG;
    if (p.M > 0) GB300_CHECK(check_operand(p.a, p.lda, p.K, p.M, p.type));
    if (p.db == p.dd || (dz && p.db == dz) || (p.z && p.db == p.z) || (p.a && p.db == p.a) ||
        (p.b && p.db == p.b))
      return GEMM_ERR_INVALID_ARG;
  }
  return GEMM_OK;
}

// Clusters that share a request's rows in the kernel for few of them: as many as one request may have
// rows, up to 16 and about a thousand in all (one without a row costs 6 ns).
int few_splits(const gemm_adapters_t& p) {
  const int64_t longest = std::max<int64_t>(1, p.M - p.requests + 1);
  return (int)std::min({(int64_t)16, std::max<int64_t>(1, 1024 / p.requests), longest});
}

// Whether a call takes it (adapters_few.cuh) rather than products over groups: by estimates of
// both, microseconds, fitted on GB300 to 1 to 256 requests of 1 to 16 rows, ranks 8 to 128, 1024^2
// to 8192^2.  The first grows with the clusters and the rows' weights, or with the rows that one cluster
// goes through: the host does not know whose the rows are, so as many as one request may
// have; the second with the inner size and the tiles, of which every request has its own.  (Microseconds a call
// through the Python binding, calls back to back, few and products, bf16, each request with an adapter of its own: 64 requests of a row, 4096 x 4096, rank 16
// 8.0, 41.8; rank 64 20.4, 40.0; 8192 x 8192, rank 128 74.6, 75.3; 256 requests, rank 16 20.7, 112.1; one request of 16 rows,
// rank 64 10.7, 22.5; 64 of two rows, rank 16 17.4, 42.2, of 65 and 63 of one 19.4, 41.6; what the choice has to
// keep from the first: 4 requests, one of 61 rows, rank 64 29.1, 22.5.)
bool few_rows(const gemm_handle* h, const gemm_adapters_t& p) {
  const int splits = few_splits(p);
  const double row = (double)p.rank * (double)(p.K + p.N);
  const double longest = (double)cdiv(p.M - std::min(p.requests, p.M) + 1, splits);
  const double few = std::max(6.0 + 0.006 * (double)(p.requests * splits) + 0.40e-6 * (double)p.M * row,
                              3.0 + longest * (1.8 + 9e-6 * row));
  const double tiles = (double)std::min(p.requests, p.M) * (double)cdiv(p.N, 128);
  const double products = 10.0 + 0.003 * (double)p.K + 1.5 / h->sm_count * tiles;
  return p.rank <= gb300::kFewRank && few < products;
}

// The kernel by the lanes that a row of `rank` elements feeds.
template <int DT>
void (*few_kernel(int64_t rank))(gb300::FewParams) {
  return rank <= 8 ? gb300::adapters_few_kernel<DT, 1> : rank <= 16 ? gb300::adapters_few_kernel<DT, 2>
         : rank <= 32 ? gb300::adapters_few_kernel<DT, 4> : gb300::adapters_few_kernel<DT, 8>;
}

// Enqueue it (h->mu held).
gemm_status_t run_few(gemm_handle* h, const gemm_adapters_t& p, struct CUstream_st* stream) {
  gb300::FewParams k{};
  k.M = (int)p.M; k.N = (int)p.N; k.K = (int)p.K; k.rank = (int)p.rank;
  k.requests = (int)p.requests; k.adapters = (int)p.adapters;
  k.offsets = p.offsets; k.index = p.index;
  k.x = p.x; k.ldx = p.ldx;
  k.a = p.A; k.lda = p.lda; k.stride_a = p.strideA;
  k.b = p.B; k.ldb = p.ldb; k.stride_b = p.strideB;
  k.scale = p.scale;
  k.r = p.r; k.ldr = p.ldr; k.r_dt = device_dt(p.r_type);
  k.d = p.d; k.ldd = p.ldd; k.d_dt = device_dt(p.d_type);
  k.in_place = p.r == p.d;
  k.splits = few_splits(p);
  h->last = gemm_config_t{};           // (no tile, no counters)
  h->counted = false;
  return launch(p.type == GEMM_F16 ? few_kernel<gb300::DT_F16>(p.rank) : few_kernel<gb300::DT_BF16>(p.rank), k,
                p.requests * k.splits * gb300::kFewCluster, gb300::kFewThreads, 0, stream,
                gb300::kFewCluster);
}

gemm_status_t check_adapters(const gemm_adapters_t& p) {
  if (!is_extent(p.M) || !is_extent(p.N) || !is_extent(p.K) || !is_extent(p.rank) ||
      !is_count(p.requests) || !is_count(p.adapters))
    return GEMM_ERR_INVALID_ARG;
  if ((p.type != GEMM_F16 && p.type != GEMM_BF16) || !is_epi_type(p.d_type) ||
      (p.r && !is_epi_type(p.r_type)))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (p.M == 0 || p.N == 0 || p.requests == 0) return GEMM_OK;
  if (!p.index) return GEMM_ERR_INVALID_ARG;
  GB300_CHECK(check_groups(p.offsets, p.index));
  if (!items_ok(p.M, p.requests, p.N) || !items_ok(p.M, p.requests, p.rank))
    return GEMM_ERR_INVALID_ARG;
  GB300_CHECK(check_operand(p.d, p.ldd, p.N, p.M, p.d_type));
  if (p.r) GB300_CHECK(check_operand(p.r, p.ldr, p.N, p.M, p.r_type));
  if (p.rank > 0 && p.adapters > 0) {
    GB300_CHECK(check_operand(p.u, p.ldu, p.rank, p.M, p.type));
    if (p.K > 0) {
      GB300_CHECK(check_operand(p.x, p.ldx, p.K, p.M, p.type));
      GB300_CHECK(check_stack(p.A, p.lda, p.K, p.rank, p.adapters, p.strideA, p.type));
    }
    GB300_CHECK(check_stack(p.B, p.ldb, p.rank, p.N, p.adapters, p.strideB, p.type));
    if (same_place(p.u, {p.x, p.A, p.B, p.r, p.d, p.offsets, p.index, p.scale}) ||
        same_place(p.d, {p.x, p.A, p.B, p.scale}))
      return GEMM_ERR_INVALID_ARG;
  }
  if (same_place(p.d, {p.offsets, p.index})) return GEMM_ERR_INVALID_ARG;
  if (!aligned_to(p.scale, 4)) return GEMM_ERR_MISALIGNED;
  if (p.r == p.d && (p.r_type != p.d_type || p.ldr != p.ldd)) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

}  // namespace

GEMM_API gemm_status_t gemm_grouped_linear_check(const gemm_grouped_linear_t* p) {
  return p ? check_grouped(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_grouped_linear(gemm_handle_t h, const gemm_grouped_linear_t* p,
                                           struct CUstream_st* stream) {
  NvtxRange range("gemm_grouped_linear");
  if (!h || !p) return GEMM_ERR_INVALID_ARG;
  GB300_CHECK(check_grouped(*p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  if (p->M == 0 || p->N == 0 || p->groups == 0) return GEMM_OK;
  const Product q = product_of(*p);
  std::lock_guard<std::mutex> guard(h->mu);
  GroupedPlan plan;
  GB300_CHECK(plan_grouped(h, q, plan));
  return run_grouped(h, q, plan, stream);
}

GEMM_API gemm_status_t gemm_grouped_linear_bwd_check(const gemm_grouped_linear_bwd_t* p) {
  return p ? check_grouped_bwd(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_grouped_linear_bwd(gemm_handle_t h, const gemm_grouped_linear_bwd_t* pp,
                                               struct CUstream_st* stream) {
  NvtxRange range("gemm_grouped_linear_bwd");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_grouped_linear_bwd_t& p = *pp;
  GB300_CHECK(check_grouped_bwd(p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  if (no_gradient(p)) return GEMM_OK;
  int64_t lddz = 0;
  const void* dz = dz_of(p, lddz);
  const bool da = p.da && p.M > 0 && p.K > 0, db = p.db && p.K > 0 && p.N > 0;
  const Product q_da = product_da(p, dz, lddz), q_db = product_db(p, dz, lddz);
  // both planned before anything is enqueued: a refused configuration changes no tensor
  GroupedPlan plan_da, plan_db, both;
  {
    std::lock_guard<std::mutex> guard(h->mu);
    if (da && db) GB300_CHECK(plan_both(h, q_da, q_db, both));
    if (!both.kern && da) GB300_CHECK(plan_grouped(h, q_da, plan_da));
    if (!both.kern && db) GB300_CHECK(plan_grouped(h, q_db, plan_db));
  }
  if (p.N > 0 && ((p.dz && p.M > 0) || p.dbias)) {
    GroupedActGrad g{};
    g.M = p.M; g.N = p.N; g.groups = p.groups;
    g.type = p.type; g.dbias_type = p.dbias_type;
    g.activation = p.activation;
    g.offsets = p.offsets;
    g.dd = p.dd; g.lddd = p.lddd;
    g.z = p.z; g.ldz = p.ldz;
    g.dz = p.dz; g.lddz = p.lddz;
    g.dbias = p.dbias;
    GB300_CHECK(grouped_act_grad(h, g, stream));
  }
  std::lock_guard<std::mutex> guard(h->mu);
  if (both.kern) return run_both(h, q_da, q_db, both, stream);
  if (da) GB300_CHECK(run_grouped(h, q_da, plan_da, stream));
  if (db) GB300_CHECK(run_grouped(h, q_db, plan_db, stream));
  return GEMM_OK;
}

GEMM_API gemm_status_t gemm_adapters_check(const gemm_adapters_t* p) {
  return p ? check_adapters(*p) : GEMM_ERR_INVALID_ARG;
}

GEMM_API gemm_status_t gemm_adapters(gemm_handle_t h, const gemm_adapters_t* pp,
                                     struct CUstream_st* stream) {
  NvtxRange range("gemm_adapters");
  if (!h || !pp) return GEMM_ERR_INVALID_ARG;
  const gemm_adapters_t& p = *pp;
  GB300_CHECK(check_adapters(p));
  if (!on_device(h)) return GEMM_ERR_INVALID_ARG;
  if (p.M == 0 || p.N == 0 || p.requests == 0) return GEMM_OK;
  const bool any = p.rank > 0 && p.adapters > 0;
  std::lock_guard<std::mutex> guard(h->mu);
  if (any && p.K > 0 && few_rows(h, p) && !h->forced) return run_few(h, p, stream);
  // (u is rounded to the operands' 16 bits: the second product's matrix units take no more)
  Product down, up;
  down.rows = p.M; down.feats = p.rank; down.k = p.K; down.groups = p.requests;
  down.sets = p.adapters;
  down.f_type = down.t_type = p.type;
  down.f = p.A; down.ldf = p.lda; down.stride_f = p.strideA;
  down.t = p.x; down.ldt = p.ldx;
  down.k_params.offsets = p.offsets; down.k_params.index = p.index;
  down.k_params.alpha = 1.f;
  down.k_params.d = p.u; down.k_params.ldd = p.ldu; down.k_params.d_dt = p.type;
  down.k_params.skip_none = 1;             // (their u is not read)
  up.rows = p.M; up.feats = p.N; up.k = any ? p.rank : 0; up.groups = p.requests;
  up.sets = p.adapters;
  up.f_type = up.t_type = p.type;
  up.f = p.B; up.ldf = p.ldb; up.stride_f = p.strideB;
  up.t = p.u; up.ldt = p.ldu;
  up.k_params.offsets = p.offsets; up.k_params.index = p.index;
  up.k_params.alpha = 1.f;
  up.k_params.set_scale = p.scale;
  up.k_params.r = p.r; up.k_params.ldr = p.ldr; up.k_params.r_dt = p.r_type;
  up.k_params.d = p.d; up.k_params.ldd = p.ldd; up.k_params.d_dt = p.d_type;
  up.k_params.skip_none = p.r == p.d;
  GroupedPlan plan_down, plan_up;
  if (any) GB300_CHECK(plan_grouped(h, down, plan_down));
  GB300_CHECK(plan_grouped(h, up, plan_up));
  if (any) GB300_CHECK(run_grouped(h, down, plan_down, stream));
  return run_grouped(h, up, plan_up, stream);
}
