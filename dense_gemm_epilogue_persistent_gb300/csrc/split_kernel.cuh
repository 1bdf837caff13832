// The linear layer for problems with too few tiles to fill the GPU (single
// tokens and decode batches, short prompts, gradients of small layers): a
// tile's K is split over the CTAs of a cluster.
//
//   D(m,n) = act(alpha row_scale(m) col_scale(n) sum_k A(m,k) B(n,k) + bias(n)) + R(m,n)
//
// Tiles are `feats` features (rows of B, the MMA's M; a multiple of 8 up to 128)
// x bn tokens (rows of A, its N, a multiple of 16): with few tokens the weights
// are what has to be read, once, and the accumulator then has a feature per
// tensor-memory lane, so a warp's accesses to D, R and Z are 32 consecutive
// elements of a row, whatever the row stride.  The MMA always spans 128 rows: with
// fewer features the rest of its rows are whatever follows in shared memory,
// and their lanes are never read; that lets the features be cut into as many
// tiles as there are SMs to stream them.  A cluster of S CTAs takes one tile, CTA r the k-blocks
// [r KB/S, (r+1) KB/S).  Each CTA's partial sums then go, by columns, to the
// CTA that owns them (distributed shared memory, the drained operand ring),
// which adds them in rank order and runs the epilogue: one launch, no
// workspace, the same bits every time.
//
// Block = 6 warps: TMA producer, tensor-memory allocator + MMA issuer, four
// epilogue warps.  Every barrier wait is bounded as in gemm_kernel.cuh; the
// cluster barriers are reached by every thread on every path.
#pragma once

#include "activations.cuh"
#include "gemm_kernel.cuh"
#include "ptx.cuh"

namespace gb300 {

struct SplitParams {
  int M, N;                  // tokens, features
  int bn;                    // tokens per tile (multiple of 16, <= 128)
  int feats;                 // features per tile (multiple of 8, <= 128)
  int ka;                    // k-blocks per ring stage
  int tiles_m;               // tiles along the tokens
  int split;                 // CTAs per cluster (S)
  int own;                   // columns a CTA owns after the exchange (multiple of 4)
  int k_blocks;              // 128-byte k-blocks
  int stages;
  int feat_mn, tok_mn;       // operand stored MN-major
  uint32_t idesc;
  uint32_t tmem_cols;        // power of two >= bn
  int inject_stall;          // test only, as in KernelParams
  uint32_t* status;
  unsigned long long timeout_ns;
  float alpha;
  const float* row_scale;
  const float* col_scale;
  const void* bias;
  const void* r;
  void* z;
  void* d;
  long long ldr, ldz, ldd;
  int bias_dt, r_dt, z_dt, d_dt;
  int act;
};

constexpr int kSplitThreads = 192;
constexpr int kSplitMaxStages = 12;

// Shared memory behind the ring: full and empty barriers, the accumulator's,
// the watchdog test's, tensor-memory address and abort flag.
constexpr uint32_t kSplitBarBytes = 8 * (2 * kSplitMaxStages + 2) + 8;

__device__ __forceinline__ float epi_load(const void* p, long long i, int dt) {
  if (dt == DT_F32) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return dt == DT_F16 ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
}

__device__ __forceinline__ void epi_store(void* p, long long i, int dt, float v) {
  if (dt == DT_F32) static_cast<float*>(p)[i] = v;
  else if (dt == DT_F16) static_cast<uint16_t*>(p)[i] = __half_as_ushort(__float2half_rn(v));
  else static_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <int AB_BYTES>
__global__ void __launch_bounds__(kSplitThreads, 1)
linear_split_kernel(const __grid_constant__ CUtensorMap tmF, const __grid_constant__ CUtensorMap tmT,
                    const __grid_constant__ SplitParams p) {
  constexpr int KIND = (AB_BYTES == 1) ? 1 : (AB_BYTES == 4 ? 2 : 0);
  constexpr int BK = 128 / AB_BYTES;             // K of a k-block
  constexpr int UMMA_K = 32 / AB_BYTES;
  constexpr int ATOM_MN = 128 / AB_BYTES;        // rows of one MN-major atom
  constexpr uint32_t ATOM_BYTES = BK * 128;      // bytes of one MN-major atom column

  grid_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // the same in every CTA of the cluster
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split;
  const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
  const int tile = blockIdx.x / S;
  const int m0 = (tile % p.tiles_m) * p.bn, n0 = (tile / p.tiles_m) * p.feats;
  const int kb0 = (int)((long long)p.k_blocks * rank / S);
  const int kb1 = (int)((long long)p.k_blocks * (rank + 1) / S);

  const uint32_t f_atom = (uint32_t)p.feats * 128u, t_atom = (uint32_t)p.bn * 128u;
  const uint32_t f_stage = f_atom * p.ka, t_stage = t_atom * p.ka;
  const uint32_t f_ring = base, t_ring = f_ring + p.stages * f_stage;
  const uint32_t bars = t_ring + p.stages * t_stage;
  const uint32_t full0 = bars, empty0 = bars + 8u * p.stages;
  const uint32_t done = empty0 + 8u * p.stages, never = done + 8u;
  const uint32_t holder = never + 8u;
  volatile uint32_t* const holder_ptr = reinterpret_cast<volatile uint32_t*>(gbase + (holder - base));
  volatile uint32_t* const abort_ptr = holder_ptr + 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    mbar_init(done, 1);
    mbar_init(never, 1);
    *abort_ptr = 0u;
    fence_barrier_init();
    prefetch_tensormap(&tmF);
    prefetch_tensormap(&tmT);
  }
  if (warp == 1) {
    tmem_alloc<1>(holder, p.tmem_cols);
    tmem_relinquish<1>();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *holder_ptr;
  // While the stream's previous kernel finishes: this CTA's first weights into
  // L2.  (A prefetch changes nothing if that kernel writes them: L2 is where its
  // writes land.)
  if (warp == 0 && !p.feat_mn && elect_one()) {
    const int n_pre = min(kb1 - kb0, p.stages * p.ka);
    for (int a = 0; a < n_pre; ++a) tma_prefetch_3d(&tmF, (kb0 + a) * BK, n0, 0);
  }
  __syncwarp();
  grid_dependency_wait();
  const Watch w{abort_ptr, p.status, p.timeout_ns};

  // The epilogue warps' state: feature n of this thread, its scale and bias.
  const int q = warp & 3;
  const int n = n0 + q * 32 + lane;
  const bool mine = n < p.N && q * 32 + lane < p.feats;
  float scale = p.alpha, bias = 0.f;
  bool ready = true;

  // The producer and the MMA warp run their loops whole, with only the
  // asynchronous instructions under the elected lane: addresses, coordinates and
  // descriptors then stay in uniform registers, where those instructions take
  // them from (1 x 8192 x 8192 bf16 on 64 CTAs: 37.7 us with the loops inside one
  // lane's branch, 28.4 us so).
  const int ka = p.ka, stages = p.stages, bn = p.bn, feats = p.feats;
  const int feat_mn = p.feat_mn, tok_mn = p.tok_mn;
  const uint32_t idesc = p.idesc;
  if (warp == 0) {
    // The features (weights) are read once; the tokens by every tile's CTAs.
    const uint64_t pol_f = make_l2_policy(2), pol_t = make_l2_policy(0);
    int s = 0;
    uint32_t ph = 0;
    for (int kb = kb0; kb < kb1; kb += ka) {
      if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(empty0 + 8u * s, ph ^ 1u, w, kWaitProducer)))
        break;
      const uint32_t fb = full0 + 8u * s;
      const int n_atoms = min(ka, kb1 - kb);
      if (elect_one()) {
        mbar_arrive_expect_tx(fb, n_atoms * (f_atom + t_atom));
        for (int a = 0; a < n_atoms; ++a) {
          const uint32_t sf = f_ring + s * f_stage + a * f_atom;
          const uint32_t st = t_ring + s * t_stage + a * t_atom;
          const int k0 = (kb + a) * BK;
          if (!feat_mn) {
            tma_load_3d(sf, &tmF, fb, k0, n0, 0, pol_f);
          } else {
            for (int j = 0; j < feats / ATOM_MN; ++j)
              tma_load_3d(sf + j * ATOM_BYTES, &tmF, fb, n0 + j * ATOM_MN, k0, 0, pol_f);
          }
          if (!tok_mn) {
            tma_load_3d(st, &tmT, fb, k0, m0, 0, pol_t);
          } else {
            for (int j = 0; j < bn / ATOM_MN; ++j)
              tma_load_3d(st + j * ATOM_BYTES, &tmT, fb, m0 + j * ATOM_MN, k0, 0, pol_t);
          }
        }
      }
      __syncwarp();
      if (++s == stages) { s = 0; ph ^= 1u; }
    }
  } else if (warp == 1) {
    // The descriptors' constant parts are built once (their address field counts
    // 16-byte units); a stage and a K step only add to them.
    const uint64_t f_desc0 = feat_mn ? smem_desc_sw128(f_ring, ATOM_BYTES, 1024)
                                       : smem_desc_sw128(f_ring, 16, 1024);
    const uint64_t t_desc0 = tok_mn ? smem_desc_sw128(t_ring, ATOM_BYTES, 1024)
                                      : smem_desc_sw128(t_ring, 16, 1024);
    const uint32_t f_step = (feat_mn ? UMMA_K * 128 : 32) / 16;
    const uint32_t t_step = (tok_mn ? UMMA_K * 128 : 32) / 16;
    int s = 0;
    uint32_t ph = 0;
    uint64_t f_desc = f_desc0, t_desc = t_desc0;
    bool ok = !p.inject_stall ||
              __all_sync(0xFFFFFFFFu, wait_phase<true>(never, 0u, w, kWaitInjected));
    for (int kb = kb0; ok && kb < kb1; kb += ka) {
      ok = __all_sync(0xFFFFFFFFu, wait_phase<true>(full0 + 8u * s, ph, w, kWaitMmaFull));
      if (!ok) break;
      tc_fence_after_sync();
      const int n_atoms = min(ka, kb1 - kb);
      if (elect_one()) {
        uint64_t fd = f_desc, td = t_desc;
        for (int a = 0; a < n_atoms; ++a) {
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k)
            umma<1, KIND>(tmem, fd + k * f_step, td + k * t_step, idesc,
                          (kb != kb0 || a != 0 || k != 0) ? 1u : 0u);
          fd += f_atom / 16;
          td += t_atom / 16;
        }
        umma_commit<1, false>(empty0 + 8u * s, 0);
        if (kb + ka >= kb1) umma_commit<1, false>(done, 0);
      }
      __syncwarp();
      f_desc += f_stage / 16;
      t_desc += t_stage / 16;
      if (++s == stages) { s = 0; ph ^= 1u; f_desc = f_desc0; t_desc = t_desc0; }
    }
  } else {
    if (mine) {
      if (p.col_scale) scale *= __ldg(p.col_scale + n);
      if (p.bias) bias = vector_elem(p.bias, n, p.bias_dt);
    }
    ready = __all_sync(0xFFFFFFFFu, wait_phase<true>(done, 0u, w, kWaitEpilogue));
    tc_fence_after_sync();
  }

  // `cols` (up to W, the length of v) columns of the tile: tokens m0 + col .., this thread's feature.  Loads
  // are issued for all of them before the first is used.
  auto finish = [&](int col, auto& v, int cols) {
    constexpr int W = sizeof(v) / sizeof(v[0]);
    const int m = m0 + col, count = mine ? min(cols, p.M - m) : 0;
    if (p.row_scale) {
      float f[W];
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = i < count ? __ldg(p.row_scale + m + i) : 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = fmaf(v[i], scale * f[i], bias);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = fmaf(v[i], scale, bias);
    }
    float r[W];
#pragma unroll
    for (int i = 0; i < W; ++i)
      r[i] = p.r && i < count ? epi_load(p.r, (m + i) * p.ldr + n, p.r_dt) : 0.f;
    if (p.z) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < count) epi_store(p.z, (m + i) * p.ldz + n, p.z_dt, v[i]);
    }
    with_activation(p.act, [&](auto a) {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = activate<decltype(a)::value>(v[i]);
    });
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < count) epi_store(p.d, (m + i) * p.ldd + n, p.d_dt, p.r ? v[i] + r[i] : v[i]);
  };
  // Columns c .. c + 15 of this warp's lanes.
  const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
  auto read_acc = [&](int c, float (&v)[16]) {
    uint32_t acc[16];
    __syncwarp();                                // (.aligned, after per-lane work)
    tmem_load_16cols(tbase + c, acc);
    tmem_wait_ld16(acc);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(acc[i]);
  };
  const bool active = warp >= 2 && ready && q * 32 < p.feats;
  if (S == 1) {
    if (active) {
      for (int c = 0; c < p.bn && m0 + c < p.M; c += 16) {
        float v[16];
        read_acc(c, v);
        if (p.M - m0 - c > 4) {
          finish(c, v, 16);
        } else {
          float u[4] = {v[0], v[1], v[2], v[3]};
          finish(c, u, 4);
        }
      }
    }
  } else {
    // Exchange: the piece of 4 columns c goes to CTA c / own, at
    // [source][piece][feature] of its drained ring.
    const int pieces = p.own / 4;                // of one owner
    cluster_sync_all();                          // every CTA's products are complete
    if (active) {
      for (int c = 0; c < p.bn; c += 16) {
        float v[16];
        read_acc(c, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int owner = (c + 4 * i) / p.own, piece = (c + 4 * i - owner * p.own) / 4;
          const uint32_t at = base + (uint32_t)((((int)rank * pieces + piece) * 128 + q * 32 + lane) * 16);
          store_cluster_v4(map_to_rank(at, (uint32_t)owner), __float_as_uint(v[4 * i]),
                           __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                           __float_as_uint(v[4 * i + 3]));
        }
      }
    }
    cluster_sync_all();                          // every partial sum has arrived
    // W columns from piece `piece` on: the sources' sums in rank order.
    auto gather = [&](int piece, auto& v) {
      constexpr int W = sizeof(v) / sizeof(v[0]);
      const int col = (int)rank * p.own + piece * 4;
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = 0.f;
      for (int src = 0; src < S; ++src) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          if (piece + i >= pieces) break;
          const float4 u = *reinterpret_cast<const float4*>(
              gbase + (size_t)(((src * pieces + piece + i) * 128 + q * 32 + lane) * 16));
          v[4 * i] += u.x; v[4 * i + 1] += u.y; v[4 * i + 2] += u.z; v[4 * i + 3] += u.w;
        }
      }
      finish(col, v, min(W, min(p.own - piece * 4, p.bn - col)));
    };
    if (active) {
      const int cols = min(p.own, min(p.bn, p.M - m0) - (int)rank * p.own);   // with tokens
      int c = 0;
      for (; c + 4 < cols; c += 16) {
        float v[16];
        gather(c / 4, v);
      }
      if (c < cols) {
        float v[4];
        gather(c / 4, v);
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (*abort_ptr) {
    // A wait gave up: let copies and MMAs already issued drain first.
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  __syncwarp();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<1>(tmem, p.tmem_cols);
  }
}

}  // namespace gb300
