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
// Block = 6 or 10 warps: TMA producer, tensor-memory allocator + MMA issuer, and
// one or two epilogue warps per lane quarter, which take its groups of columns in
// turn (128 x 512 x 512 E4M3 7.9 us with two, 8.9 with one; 1 x 4096 x 4096 bf16 9.4
// and 9.1: two from 17 tokens on).  Every barrier wait is bounded as in gemm_kernel.cuh; the
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
  int trigger_late, wait_late;   // as in EpiParams
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

constexpr int kSplitThreads = 320;           // at most: 192 with four epilogue warps
constexpr int kSplitMaxStages = 12;

// Shared memory behind the ring: full and empty barriers, the accumulator's,
// the watchdog test's, tensor-memory address and abort flag.
constexpr uint32_t kSplitBarBytes = 8 * (2 * kSplitMaxStages + 2) + 8;

__device__ __forceinline__ int epi_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }

// Elements of `count` (up to 4) rows `step` bytes apart.
__device__ __forceinline__ void epi_store4(uint8_t* p, long long step, int dt, int count,
                                           const float4& v) {
  if (dt == DT_F32) {
    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) *reinterpret_cast<float*>(p + i * step) = e[i];
  } else {
    const uint32_t w[2] = {dt == DT_F16 ? pack_f16x2(v.x, v.y) : pack_bf16x2(v.x, v.y),
                           dt == DT_F16 ? pack_f16x2(v.z, v.w) : pack_bf16x2(v.z, v.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count)
        *reinterpret_cast<uint16_t*>(p + i * step) = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}

// One copy of the activations' code, called: the epilogue runs each line of
// its own code once or a few times, so that fetching it costs more than a call.
template <int AB_BYTES>
__device__ __noinline__ float4 activate4(float4 v, int act) {
  with_activation(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    activate2<ACT>(v.x, v.y);
    activate2<ACT>(v.z, v.w);
  });
  return v;
}

template <int AB_BYTES>
__global__ void __launch_bounds__(kSplitThreads, 2)
linear_split_kernel(const __grid_constant__ CUtensorMap tmF, const __grid_constant__ CUtensorMap tmT,
                    const __grid_constant__ SplitParams p) {
  constexpr int KIND = (AB_BYTES == 1) ? 1 : (AB_BYTES == 4 ? 2 : 0);
  constexpr int BK = 128 / AB_BYTES;             // K of a k-block
  constexpr int UMMA_K = 32 / AB_BYTES;
  constexpr int ATOM_MN = 128 / AB_BYTES;        // rows of one MN-major atom
  constexpr uint32_t ATOM_BYTES = BK * 128;      // bytes of one MN-major atom column

  if (!p.trigger_late) grid_launch_dependents();
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
  if (!p.wait_late) grid_dependency_wait();
  if (p.trigger_late) grid_launch_dependents();
  const Watch w{abort_ptr, p.status, p.timeout_ns};

  // The epilogue warps' state: feature n of this thread, its scale and bias.
  const int q = warp & 3, turn = (warp - 2) >> 2, turns = ((int)blockDim.x - 64) >> 7;
  const int n = n0 + q * 32 + lane;
  const bool mine = n < p.N && q * 32 + lane < p.feats;
  float scale = p.alpha, bias = 0.f;
  bool ready = true;
  // The columns this CTA finishes: [c_lo, c_lo + n_cols) of the tile, those of
  // its share that hold tokens, four at a time, every `turns`-th four this warp's.
  // Residuals of its first four groups are fetched while the main loop runs,
  // then four groups ahead; a lane holds one column's row factor of 32.
  const int with_tokens = min(p.bn, p.M - m0);
  const int c_lo = S > 1 ? (int)rank * p.own : 0;
  const int n_cols = max(0, min(S > 1 ? p.own : p.bn, with_tokens - c_lo));
  const long long m_lo = m0 + c_lo;
  const long long d_step = p.ldd * epi_bytes(p.d_dt), r_step = p.ldr * epi_bytes(p.r_dt);
  const long long z_step = p.ldz * epi_bytes(p.z_dt);
  uint8_t* d_at = static_cast<uint8_t*>(p.d) + m_lo * d_step + (long long)n * epi_bytes(p.d_dt);
  uint8_t* z_at = static_cast<uint8_t*>(p.z) + m_lo * z_step + (long long)n * epi_bytes(p.z_dt);
  const uint8_t* r_at =
      static_cast<const uint8_t*>(p.r) + m_lo * r_step + (long long)n * epi_bytes(p.r_dt);
  // (as they lie in memory: converted where they are used, so that a fetch
  // waits for nothing)
  uint32_t r[16];
  auto fetch = [&](int g, int c) {               // r[4 g ..] for columns c ..
    const uint8_t* const at = r_at + c * r_step;
    if (p.r_dt == DT_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[4 * g + i] = mine && c + i < n_cols
                           ? *reinterpret_cast<const uint32_t*>(at + i * r_step) : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[4 * g + i] = mine && c + i < n_cols
                           ? *reinterpret_cast<const uint16_t*>(at + i * r_step) : 0u;
    }
  };
  auto residual = [&](uint32_t bits) {
    return p.r_dt == DT_F32   ? __uint_as_float(bits)
           : p.r_dt == DT_F16 ? __half2float(__ushort_as_half((uint16_t)bits))
                              : __uint_as_float(bits << 16);
  };
  auto row_factor = [&](int c) {                 // this lane's of columns c .. c + 31
    return p.row_scale && c + lane < n_cols ? __ldg(p.row_scale + m_lo + c + lane) : 1.f;
  };
  float factor = 1.f, next_factor = 1.f;

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
      // (debug build, by every lane alike: the boxes inside this stage, their inner
      // coordinates whole 16 bytes, all from 0 on)
      if (!dbg_check(in_range(f_ring + s * f_stage, n_atoms * f_atom, f_ring, t_ring) &&
                         in_range(t_ring + s * t_stage, n_atoms * t_atom, t_ring, bars) &&
                         n0 >= 0 && m0 >= 0 && (!feat_mn || n0 * AB_BYTES % 16 == 0) &&
                         (!tok_mn || m0 * AB_BYTES % 16 == 0),
                     kChkLoadA, w))
        break;
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
      // (debug build: the accumulator's columns allocated, the operands' start addresses
      // inside the stage, and 128 rows of features inside the block's memory)
      if constexpr (kDebug) {
        ok = dbg_check((uint32_t)bn <= p.tmem_cols && p.tmem_cols <= kTmemCols, kChkMmaTmem, w);
        for (int a = 0; a < n_atoms; ++a) {
          const uint32_t fa = f_ring + s * f_stage + a * f_atom, ta = t_ring + s * t_stage + a * t_atom;
          for (int k = 0; k < BK / UMMA_K; ++k)
            ok = ok && dbg_check(desc_in_range(f_desc + a * (f_atom / 16) + k * f_step, fa, f_atom) &&
                                     desc_in_range(t_desc + a * (t_atom / 16) + k * t_step, ta,
                                                   t_atom) &&
                                     fa + 128u * 128u <= raw + dynamic_smem_bytes(),
                                 kChkMmaSmem, w);
        }
        if (!ok) break;
      }
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
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (p.r && 4 * (g * turns + turn) < n_cols) fetch(g, 4 * (g * turns + turn));
    next_factor = row_factor(0);
    ready = __all_sync(0xFFFFFFFFu, wait_phase<true>(done, 0u, w, kWaitEpilogue));
    tc_fence_after_sync();
  }

  const bool active = warp >= 2 && ready && q * 32 < p.feats;
  const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
  // Partial sums by pieces of 4 columns: [source][piece of its owner][feature].
  const int pieces = p.own / 4;
  const uint32_t my_piece = (uint32_t)(q * 32 + lane) * 16u;
  if (S > 1) {
    cluster_sync_all();                          // every CTA's products are complete
    if (active) {
      int owner = 0, piece = 0;
      auto advance = [&](int n_pieces) {
        piece += n_pieces;
        while (piece >= pieces) { piece -= pieces; ++owner; }
      };
      advance(4 * turn);
      for (int c = 16 * turn; c < with_tokens; c += 16 * turns) {
        uint32_t acc[16];
        // (debug build: the columns allocated, each piece inside its owner's ring)
        if (!dbg_check((uint32_t)c + 16u <= p.tmem_cols, kChkEpiTmem, w)) break;
        __syncwarp();
        tmem_load_16cols(tbase + c, acc);
        tmem_wait_ld16(acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c + 4 * i < with_tokens &&
              dbg_check(owner < S && in_range(base + (rank * pieces + piece) * 2048u + my_piece, 16,
                                              base, bars),
                        kChkEpiSmem, w))
            store_cluster_v4(map_to_rank(base + (rank * pieces + piece) * 2048u + my_piece,
                                         (uint32_t)owner),
                             acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
          advance(1);
        }
        advance(4 * (turns - 1));
      }
    }
    cluster_sync_all();                          // every partial sum has arrived
  }
  if (active) {
    // (not unrolled: the body runs once or a few times, from instruction lines
    // nothing has fetched yet)
    z_at += 4 * turn * z_step;
    d_at += 4 * turn * d_step;
#pragma unroll 1
    for (int c = 4 * turn; c < n_cols; c += 4 * turns) {
      if ((c & 31) < 4 * turns) {                        // (the warp's first group of 32)
        factor = next_factor;
        next_factor = row_factor((c & ~31) + 32);
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      // (debug build: accumulator columns allocated or pieces inside the ring; the stores
      // below inside D)
      if (!dbg_check(S == 1 ? (uint32_t)c + 4u <= p.tmem_cols
                            : in_range(base + c * 512 + ((S - 1) * pieces) * 2048u + q * 512u, 512u,
                                       base, bars),
                     kChkEpiSmem, w) ||
          !dbg_check(n0 >= 0 && m_lo >= 0 && m_lo + n_cols <= p.M, kChkEpiStore, w))
        break;
      if (S == 1) {
        uint32_t acc[4];
        __syncwarp();                            // (.aligned, after per-lane work)
        tmem_load_4cols(tbase + c, acc);
        tmem_wait_ld4(acc);
        v = make_float4(__uint_as_float(acc[0]), __uint_as_float(acc[1]), __uint_as_float(acc[2]),
                        __uint_as_float(acc[3]));
      } else {
        const uint8_t* at = gbase + c * 512 + my_piece;
#pragma unroll 2
        for (int src = 0; src < S; ++src, at += pieces * 2048) {
          const float4 u = *reinterpret_cast<const float4*>(at);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
      }
      v.x = fmaf(v.x, scale * __shfl_sync(0xFFFFFFFFu, factor, c & 31), bias);
      v.y = fmaf(v.y, scale * __shfl_sync(0xFFFFFFFFu, factor, (c + 1) & 31), bias);
      v.z = fmaf(v.z, scale * __shfl_sync(0xFFFFFFFFu, factor, (c + 2) & 31), bias);
      v.w = fmaf(v.w, scale * __shfl_sync(0xFFFFFFFFu, factor, (c + 3) & 31), bias);
      const int count = mine ? n_cols - c : 0;
      if (p.z) {
        epi_store4(z_at, z_step, p.z_dt, count, v);
        z_at += 4 * turns * z_step;
      }
      if (p.act != ACT_NONE) v = activate4<AB_BYTES>(v, p.act);
      if (p.r) {
        v.x += residual(r[0]);
        v.y += residual(r[1]);
        v.z += residual(r[2]);
        v.w += residual(r[3]);
#pragma unroll
        for (int i = 0; i < 12; ++i) r[i] = r[i + 4];
        if (c + 16 * turns < n_cols) fetch(3, c + 16 * turns);
      }
      epi_store4(d_at, d_step, p.d_dt, count, v);
      d_at += 4 * turns * d_step;
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
  if (p.wait_late) grid_dependency_wait();
}

}  // namespace gb300
