// ssa_mass.cu -- attention weight that each cached key received
// (ssa_attn_mass) on B200 (sm_100a).
//
// Given the rows' log-sum-exp, the weight of key j is a sum over query rows of
// exp(scale q.k_j - lse).  Both kernels compute S^T = K Q^T on tcgen05 with the
// 128 keys of a tile on the M side, so that a TMEM lane is a key: one thread owns
// a key and adds its row's exponentials in registers, with no reduction between
// threads, no atomics and no probabilities written anywhere.  Query rows are
// packed token-major over the G query heads of a key head (row i * G + g).
//
//   stream kernel: all G * window rows fit one operand tile (<= 256 rows).  The
//     rows stay in shared memory and the key tiles stream past, each read
//     once: bound by HBM (2 * d bytes a key and key head).
//   prompt kernel: more rows.  A key tile stays and the row tiles stream past
//     from L2: bound by the exponentials (MUFU, 16 a clock and SM: 1,024
//     clocks a 128 x 128 tile against 512 for its matrix product).
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/ssa_cache.h"
#include "internal.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace ssa_mass {

namespace cg = cooperative_groups;
using ssa::clamp_len;
using ssa::mbar_arrive;
using ssa::mbar_arrive_expect_tx;
using ssa::mbar_init;
using ssa::Seg;
using ssa::SegWalk;
using ssa::smem_u32;

constexpr int BK = 128;  // keys per tile: the M of the MMA
constexpr int NT = 384;  // warp 0 producer, 1 MMA, 2 rows and lse, 3 zero fill, 4-11 sums
constexpr unsigned long long DRAIN_NS = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f;

struct Params {
  const float* lse;
  const float* mass_in;
  float* mass_out;
  const int32_t* lens;
  int* status;
  unsigned long long wait_ns;
  int B, Lq, W, Hq, Hkv, G, cap, causal;
  float c;  // scale * log2(e)
  float decay;
  int tok, tiles;  // prompt kernel: tokens per row tile, row tiles
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// -lse in log2 units; a row without keys (-inf) and a row that is not there get
// -inf, so that their exponentials are 0
__device__ __forceinline__ float neg_lse2(const Params& p, int b, int hkv, int r) {
  const int i = p.Lq - p.W + r / p.G;
  if (i >= p.Lq) return -INFINITY;
  const float l = p.lse[((size_t)b * p.Hq + hkv * p.G + r % p.G) * p.Lq + i];
  return l == -INFINITY ? -INFINITY : -l * LOG2E;
}

// Adds exp2(s c + nl) over NC columns; columns below `first` do not count.
template <int NC, bool MASK>
__device__ __forceinline__ void add_columns(const float* x, const float* nl, float c, int first, uint64_t (&acc)[2]) {
  const uint64_t c2 = ssa::f2_pack(c, c);
#pragma unroll
  for (int i = 0; i < NC; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(nl + i);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t e = ssa::ffma2(ssa::f2_pack(x[i + 2 * h], x[i + 2 * h + 1]), c2,
                                    h ? ssa::f2_pack(l.z, l.w) : ssa::f2_pack(l.x, l.y));
      float e0, e1;
      ssa::f2_unpack(e, e0, e1);
      float p0 = ex2(e0), p1 = ex2(e1);
      if (MASK) {
        p0 = i + 2 * h >= first ? p0 : 0.f;
        p1 = i + 2 * h + 1 >= first ? p1 : 0.f;
      }
      acc[h] = ssa::fadd2(acc[h], ssa::f2_pack(p0, p1));
    }
  }
}
__device__ __forceinline__ float total(const uint64_t (&acc)[2]) {
  float a, b, c, d;
  ssa::f2_unpack(acc[0], a, b);
  ssa::f2_unpack(acc[1], c, d);
  return (a + b) + (c + d);
}

template <int NC>
__device__ __forceinline__ void load_columns(uint32_t taddr, float* x) {
  if constexpr (NC == 16) ssa::tmem_ld16f(taddr, x);
  else if constexpr (NC == 32) ssa::tmem_ld32f(taddr, x);
  else ssa::tmem_ld64f(taddr, x);
}

// ============================================================ stream kernel

template <int D, int N>
struct StreamSmem {
  static constexpr uint32_t Q_BYTES = N * D * 2;
  static constexpr uint32_t K_BYTES = BK * D * 2;
  static constexpr int FIT = (int)((208 * 1024 - Q_BYTES) / K_BYTES);
  static constexpr int KST = FIT < 8 ? FIT : 8;
  static constexpr uint32_t TOTAL = 1024 + Q_BYTES + KST * K_BYTES;
};

template <int D, int N>
__global__ void __launch_bounds__(NT, 1)
    mass_stream_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ Params p) {
  using L = StreamSmem<D, N>;
  constexpr int KST = L::KST;
  constexpr int NC = N < 64 ? N : 64;  // columns per TMEM load
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t kfull[KST], kempty[KST], q_full, q_empty, lse_full[2], lse_empty[2], s_full[2], s_empty[2], done;
  __shared__ __align__(16) float nlse[2][N];
  __shared__ int pref[ssa::MAX_SEQS + 1];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_s = smem_u32(base), k_s = q_s + L::Q_BYTES;

  if (tid == 0) {
    for (int i = 0; i < KST; ++i) {
      mbar_init(smem_u32(&kfull[i]), 1);
      mbar_init(smem_u32(&kempty[i]), 1);
    }
    mbar_init(smem_u32(&q_full), 1);
    mbar_init(smem_u32(&q_empty), 1);
    mbar_init(smem_u32(&done), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&lse_full[i]), 32);
      mbar_init(smem_u32(&lse_empty[i]), 8);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), 4);
    }
    abort_flag = 0;
    ssa::fence_mbar_init();
  }
  if (warp == 1) {
    ssa::tmem_alloc(smem_u32(&tmem_base), 512);
    ssa::tmem_relinquish();
  }
  if (warp == 2)
    ssa::tile_prefix(pref, p.B, [&](int b) { return (clamp_len(p.lens, b, p.cap) + BK - 1) / BK; });
  // operand rows past G * W are never loaded: zero
  for (int e = tid; e < (int)(L::Q_BYTES / 16); e += NT)
    reinterpret_cast<uint4*>(base)[e] = make_uint4(0u, 0u, 0u, 0u);
  ssa::fence_proxy_async_smem();
  ssa::tc_fence_before();
  __syncthreads();
  ssa::tc_fence_after();
  const uint32_t tmem = tmem_base;
  const ssa::Waiter wait{&abort_flag, p.status, p.wait_ns};
  SegWalk walk(pref, p.B, p.Hkv, blockIdx.x, gridDim.x);
  Seg s;

  if (warp == 0) {
    if (lane == 0) {
      ssa::tma_prefetch_desc(&tm_k);
      int g = 0;
      bool ok = true;
      while (ok && walk.next(s))
        for (int t = 0; t < s.nt; ++t, ++g) {
          const int st = g % KST;
          if (!wait(&kempty[st], ((g / KST) & 1) ^ 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(smem_u32(&kfull[st]), L::K_BYTES);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            ssa::tma_load_4d(k_s + st * L::K_BYTES + c * BK * 128, &tm_k, smem_u32(&kfull[st]), c * 64, s.in,
                             (s.kt0 + t) * BK, s.b);
        }
      for (int t = max(0, g - KST); t < g; ++t)  // nothing in flight when the block ends
        ssa::mbar_wait(smem_u32(&kfull[t % KST]), (t / KST) & 1, DRAIN_NS);
    }
  } else if (warp == 1) {
    {
      const uint32_t leader = ssa::elect_one();
      auto waits = [&](const uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
      constexpr uint32_t idesc = ssa::idesc_bf16_f32(BK, N, false, false);
      int g = 0, n = 0;
      bool ok = true;
      while (ok && walk.next(s)) {
        ok = waits(&q_full, n & 1);
        for (int t = 0; ok && t < s.nt; ++t, ++g) {
          const int st = g % KST;
          if (!waits(&kfull[st], (g / KST) & 1) || !waits(&s_empty[g & 1], ((g >> 1) & 1) ^ 1)) {
            ok = false;
            break;
          }
          ssa::tc_fence_after();
#pragma unroll
          for (int k16 = 0; k16 < D / 16; ++k16) {
            const uint32_t in = (k16 & 3) * 32;
            ssa::mma_ss_warp(leader, tmem + 256 * (g & 1),
                        ssa::smem_desc_sw128(k_s + st * L::K_BYTES + (k16 >> 2) * BK * 128 + in, 16, 1024),
                        ssa::smem_desc_sw128(q_s + (k16 >> 2) * N * 128 + in, 16, 1024), idesc, k16 > 0);
          }
          ssa::mma_commit_warp(leader, smem_u32(&s_full[g & 1]));
          ssa::mma_commit_warp(leader, smem_u32(&kempty[st]));
        }
        if (ok) ssa::mma_commit_warp(leader, smem_u32(&q_empty));
        ++n;
      }
      ssa::mma_commit_warp(leader, smem_u32(&done));
      ssa::mbar_wait(smem_u32(&done), 0, DRAIN_NS);  // no MMA in flight when TMEM is freed
    }
  } else if (warp == 2) {
    int n = 0;
    while (walk.next(s)) {
      bool ok = wait(&lse_empty[n & 1], ((n >> 1) & 1) ^ 1) && wait(&q_empty, (n & 1) ^ 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&q_full), (uint32_t)(p.G * p.W * D * 2));
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          ssa::tma_load_4d(q_s + c * N * 128, &tm_q, smem_u32(&q_full), c * 64, s.in * p.G, p.Lq - p.W, s.b);
      }
      for (int r = lane; r < N; r += 32)
        nlse[n & 1][r] = r < p.G * p.W ? neg_lse2(p, s.b, s.in, r) : -INFINITY;
      mbar_arrive(smem_u32(&lse_full[n & 1]));
      ++n;
    }
    if (n > 0 && lane == 0) ssa::mbar_wait(smem_u32(&q_full), (n - 1) & 1, DRAIN_NS);
  } else if (warp == 3) {
    // keys past each sequence's last tile: no weight
    for (int x = blockIdx.x; x < p.B * p.Hkv; x += gridDim.x) {
      const int n = clamp_len(p.lens, x / p.Hkv, p.cap);
      for (int j = (n + BK - 1) / BK * BK + lane; j < p.cap; j += 32) p.mass_out[(size_t)x * p.cap + j] = 0.f;
    }
  } else {
    const int wg = (warp - 4) >> 2;  // tiles wg, wg + 2, ...
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256 * wg;
    const int row = (warp & 3) * 32 + lane;
    int g = 0, n = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const int len = clamp_len(p.lens, s.b, p.cap);
      const size_t out = ((size_t)s.b * p.Hkv + s.in) * p.cap;
      ok = __all_sync(0xffffffffu, wait(&lse_full[n & 1], (n >> 1) & 1));
      for (int t = 0; ok && t < s.nt; ++t, ++g) {
        if ((g & 1) != wg) continue;
        const int j0 = (s.kt0 + t) * BK, j = j0 + row;
        const float before = p.mass_in != nullptr && j < len ? p.decay * p.mass_in[out + j] : 0.f;
        ok = __all_sync(0xffffffffu, wait(&s_full[wg], (g >> 1) & 1));
        if (!ok) break;
        ssa::tc_fence_after();
        // row i of the window sits at i + len - W: key j counts from there on
        const bool mask = p.causal && j0 + BK - 1 > len - p.W;
        const int first = mask ? (j - len + p.W) * p.G : 0;
        uint64_t acc[2] = {ssa::f2_pack(0.f, 0.f), ssa::f2_pack(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < N / NC; ++c) {
          float x[NC];
          load_columns<NC>(lanes + c * NC, x);
          ssa::tmem_wait_ld();
          if (c == N / NC - 1) {  // S is in registers: the buffer is free
            ssa::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_empty[wg]));
          }
          if (mask) add_columns<NC, true>(x, &nlse[n & 1][c * NC], p.c, first - c * NC, acc);
          else add_columns<NC, false>(x, &nlse[n & 1][c * NC], p.c, 0, acc);
        }
        if (j < p.cap) p.mass_out[out + j] = j < len ? before + total(acc) : 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&lse_empty[n & 1]));
      ++n;
    }
  }
  ssa::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ssa::tc_fence_after();
    ssa::tmem_dealloc(tmem, 512);
  }
}

// ============================================================ prompt kernel

constexpr int BN = 128;   // rows per row tile
constexpr int NLSE = 8;   // row tiles whose lse is in shared memory
constexpr int NBUF = 4;   // S^T buffers in TMEM

template <int D>
struct PromptSmem {
  static constexpr uint32_t K_BYTES = BK * D * 2;
  static constexpr uint32_t Q_BYTES = BN * D * 2;
  static constexpr int QST = D == 128 ? 5 : 8;
  static constexpr uint32_t TOTAL = 1024 + K_BYTES + QST * Q_BYTES;
};

// Block (cluster rank r of S): key tile kt of one (sequence, key head), every
// S-th part of the row tiles that see it; the parts are added through
// distributed shared memory in rank order.
template <int D>
__global__ void __launch_bounds__(NT, 1)
    mass_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ Params p) {
  using L = PromptSmem<D>;
  constexpr int QST = L::QST;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t k_full, qfull[QST], qempty[QST], lse_full[NLSE], lse_empty[NLSE], s_full[NBUF], s_empty[NBUF], done;
  __shared__ __align__(16) float nlse[NLSE][BN];
  __shared__ float part[2][BK];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // low key tiles first: under a causal mask they are seen by the most rows
  const int item = blockIdx.x / S, pairs = p.B * p.Hkv;
  const int kt = item / pairs, pair = item % pairs;
  const int b = pair / p.Hkv, hkv = pair % p.Hkv;
  const int len = clamp_len(p.lens, b, p.cap);
  const int j0 = kt * BK;
  float* out = p.mass_out + (size_t)pair * p.cap;
  const float* in = p.mass_in != nullptr ? p.mass_in + (size_t)pair * p.cap : nullptr;
  if (j0 >= len) {  // the same for every block of the cluster
    if (rank == 0 && tid < BK && j0 + tid < p.cap) out[j0 + tid] = 0.f;
    return;
  }
  // first row tile that sees the tile's first key, and this rank's range
  const int t_first = p.causal ? min(max((j0 - len + p.W) / p.tok, 0), p.tiles) : 0;
  const int nt = p.tiles - t_first;
  const int t0 = t_first + (int)((long long)nt * rank / S), t1 = t_first + (int)((long long)nt * (rank + 1) / S);
  const uint32_t k_s = smem_u32(base), q_s = k_s + L::K_BYTES;

  if (tid == 0) {
    mbar_init(smem_u32(&k_full), 1);
    mbar_init(smem_u32(&done), 1);
    for (int i = 0; i < QST; ++i) {
      mbar_init(smem_u32(&qfull[i]), 1);
      mbar_init(smem_u32(&qempty[i]), 1);
    }
    for (int i = 0; i < NLSE; ++i) {
      mbar_init(smem_u32(&lse_full[i]), 64);
      mbar_init(smem_u32(&lse_empty[i]), 4);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), 4);
    }
    abort_flag = 0;
    ssa::fence_mbar_init();
  }
  if (warp == 1) {
    ssa::tmem_alloc(smem_u32(&tmem_base), 512);
    ssa::tmem_relinquish();
  }
  if (p.G * p.tok < BN) {  // operand rows past the tile's tokens are never loaded: zero
    for (int e = tid; e < (int)(QST * L::Q_BYTES / 16); e += NT)
      reinterpret_cast<uint4*>(base + L::K_BYTES)[e] = make_uint4(0u, 0u, 0u, 0u);
  }
  ssa::fence_proxy_async_smem();
  ssa::tc_fence_before();
  __syncthreads();
  ssa::tc_fence_after();
  const uint32_t tmem = tmem_base;
  const ssa::Waiter wait{&abort_flag, p.status, p.wait_ns};

  if (warp == 0) {
    if (lane == 0 && t0 < t1) {
      mbar_arrive_expect_tx(smem_u32(&k_full), L::K_BYTES);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        ssa::tma_load_4d(k_s + c * BK * 128, &tm_k, smem_u32(&k_full), c * 64, hkv, j0, b);
      int g = 0;
      for (int t = t0; t < t1; ++t, ++g) {
        const int st = g % QST;
        if (!wait(&qempty[st], ((g / QST) & 1) ^ 1)) break;
        mbar_arrive_expect_tx(smem_u32(&qfull[st]), (uint32_t)(p.G * p.tok * D * 2));
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          ssa::tma_load_4d(q_s + st * L::Q_BYTES + c * BN * 128, &tm_q, smem_u32(&qfull[st]), c * 64, hkv * p.G,
                           p.Lq - p.W + t * p.tok, b);
      }
      ssa::mbar_wait(smem_u32(&k_full), 0, DRAIN_NS);
      for (int t = max(0, g - QST); t < g; ++t)
        ssa::mbar_wait(smem_u32(&qfull[t % QST]), (t / QST) & 1, DRAIN_NS);
    }
  } else if (warp == 1) {
    if (t0 < t1) {
      const uint32_t leader = ssa::elect_one();
      auto waits = [&](const uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
      constexpr uint32_t idesc = ssa::idesc_bf16_f32(BK, BN, false, false);
      bool ok = waits(&k_full, 0);
      for (int g = 0; ok && g < t1 - t0; ++g) {
        const int st = g % QST, buf = g % NBUF;
        if (!waits(&qfull[st], (g / QST) & 1) || !waits(&s_empty[buf], ((g / NBUF) & 1) ^ 1)) break;
        ssa::tc_fence_after();
#pragma unroll
        for (int k16 = 0; k16 < D / 16; ++k16) {
          const uint32_t o = (k16 >> 2) * 128 * 128 + (k16 & 3) * 32;
          ssa::mma_ss_warp(leader, tmem + 128 * buf, ssa::smem_desc_sw128(k_s + o, 16, 1024),
                      ssa::smem_desc_sw128(q_s + st * L::Q_BYTES + o, 16, 1024), idesc, k16 > 0);
        }
        ssa::mma_commit_warp(leader, smem_u32(&s_full[buf]));
        ssa::mma_commit_warp(leader, smem_u32(&qempty[st]));
      }
      ssa::mma_commit_warp(leader, smem_u32(&done));
      ssa::mbar_wait(smem_u32(&done), 0, DRAIN_NS);
    }
  } else if (warp < 4) {
    const int t64 = tid - 64;
    for (int g = 0; g < t1 - t0; ++g) {
      const int sl = g % NLSE;
      if (!__all_sync(0xffffffffu, wait(&lse_empty[sl], ((g / NLSE) & 1) ^ 1))) break;
      for (int r = t64; r < BN; r += 64)
        nlse[sl][r] = r < p.G * p.tok ? neg_lse2(p, b, hkv, (t0 + g) * p.tok * p.G + r) : -INFINITY;
      mbar_arrive(smem_u32(&lse_full[sl]));
    }
  } else {
    const int wg = (warp - 4) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int row = (warp & 3) * 32 + lane, j = j0 + row;
    float sum = 0.f;
    for (int g = wg; g < t1 - t0; g += 2) {
      const int buf = g % NBUF, sl = g % NLSE;
      if (!__all_sync(0xffffffffu, wait(&lse_full[sl], (g / NLSE) & 1) && wait(&s_full[buf], (g / NBUF) & 1))) break;
      ssa::tc_fence_after();
      const int i0 = (t0 + g) * p.tok;  // the tile's first row, in the window
      const bool mask = p.causal && j0 + BK - 1 > i0 + len - p.W;
      const int first = mask ? (j - len + p.W - i0) * p.G : 0;
      uint64_t acc[2] = {ssa::f2_pack(0.f, 0.f), ssa::f2_pack(0.f, 0.f)};
      float x[BN];
      ssa::tmem_ld64f(lanes + 128 * buf, x);
      ssa::tmem_ld64f(lanes + 128 * buf + 64, x + 64);
      ssa::tmem_wait_ld();
      ssa::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_empty[buf]));
      if (mask) add_columns<BN, true>(x, nlse[sl], p.c, first, acc);
      else add_columns<BN, false>(x, nlse[sl], p.c, 0, acc);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&lse_empty[sl]));
      sum += total(acc);
    }
    part[wg][row] = sum;
  }
  ssa::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ssa::tc_fence_after();
    ssa::tmem_dealloc(tmem, 512);
  }
  if (tid < BK) part[0][tid] += part[1][tid];
  if (S > 1) cluster.sync();
  else __syncthreads();
  if (rank == 0 && tid < BK && j0 + tid < p.cap) {
    float sum = 0.f;
    for (int r = 0; r < S; ++r) sum += *cluster.map_shared_rank(&part[0][tid], r);
    const int j = j0 + tid;
    out[j] = j < len ? (in != nullptr ? p.decay * in[j] + sum : sum) : 0.f;
  }
  if (S > 1) cluster.sync();  // rank 0 still reads the others' sums
}

template <class Kernel>
static int launch(Kernel* kernel, size_t smem, long long grid, int cluster, const CUtensorMap& q, const CUtensorMap& k,
                  const Params& p, cudaStream_t st) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SSA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, q, k, p) == cudaSuccess ? SSA_OK : SSA_ERR_CUDA;
}

template <int D>
static int run(const Params& p, const void* q, const void* k, int sms, cudaStream_t st) {
  CUtensorMap mq, mk;
  if (!ssa::tma_map_bf16(&mk, k, p.B, p.cap, p.Hkv, D, BK)) return SSA_ERR_CUDA;
  const long long R = (long long)p.G * p.W, nk = ((long long)p.cap + BK - 1) / BK, pairs = (long long)p.B * p.Hkv;
  if (R <= 256) {
    if (!ssa::tma_map_bf16_box(&mq, q, p.B, p.Lq, p.Hq, D, p.G, p.W)) return SSA_ERR_CUDA;
    const long long grid = pairs * nk < sms ? pairs * nk : sms;
#define SSA_STREAM(N) launch(mass_stream_kernel<D, N>, StreamSmem<D, N>::TOTAL, grid, 1, mq, mk, p, st)
    if (R <= 16) return SSA_STREAM(16);
    if (R <= 32) return SSA_STREAM(32);
    if (R <= 64) return SSA_STREAM(64);
    if (R <= 128) return SSA_STREAM(128);
    return SSA_STREAM(256);
#undef SSA_STREAM
  }
  if (!ssa::tma_map_bf16_box(&mq, q, p.B, p.Lq, p.Hq, D, p.G, p.tok)) return SSA_ERR_CUDA;
  // few key tiles: a cluster shares one, as long as the GPU holds them all at once
  int cs = 1;
  while (cs < 8 && pairs * nk * cs * 2 <= sms && p.tiles >= cs * 4) cs *= 2;
  const long long grid = pairs * nk * cs;
  if (grid > 0x7fffffff) return SSA_ERR_UNSUPPORTED;
  return launch(mass_prompt_kernel<D>, PromptSmem<D>::TOTAL, grid, cs, mq, mk, p, st);
}

}  // namespace ssa_mass

extern "C" int ssa_attn_mass(const void* q, const void* k, const float* lse, const int32_t* lens,
                             const float* mass_in, float* mass_out, int B, int Lq, int window, int Hq, int Hkv,
                             int cap, int d, int causal, float scale, float decay, void* stream) {
  using namespace ssa_mass;
  if (!q || !k || !lse || !mass_out) return SSA_ERR_INVALID_ARG;
  if (B <= 0 || Lq <= 0 || window < 0 || window > Lq || Hq <= 0 || Hkv <= 0 || cap <= 0 || d <= 0)
    return SSA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return SSA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SSA_ERR_INVALID_ARG;
  if (mass_in && (!(decay >= 0.f) || !std::isfinite(decay))) return SSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k)) & 15u) return SSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(mass_in) |
       reinterpret_cast<uintptr_t>(mass_out)) & 3u)
    return SSA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSA_ERR_UNSUPPORTED;
  if (B > ssa::MAX_SEQS || Hq / Hkv > BN) return SSA_ERR_UNSUPPORTED;
  if ((long long)B * Hkv > (1 << 24) || (long long)Lq * Hq > 0x7fffffff || cap > (1 << 30)) return SSA_ERR_UNSUPPORTED;
  Params p{};
  p.lse = lse;
  p.mass_in = mass_in;
  p.mass_out = mass_out;
  p.lens = lens;
  p.B = B;
  p.Lq = Lq;
  p.W = window > 0 ? window : Lq;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.cap = cap;
  p.causal = causal ? 1 : 0;
  p.c = (float)((double)scale * 1.4426950408889634);
  p.decay = decay;
  p.tok = BN / p.G;
  p.tiles = (p.W + p.tok - 1) / p.tok;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return SSA_ERR_CUDA;
  p.status = ssa::device_status_word(dev);
  if (!p.status) return SSA_ERR_CUDA;
  p.wait_ns = ssa::wait_timeout_ns();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? run<128>(p, q, k, sms, st) : run<64>(p, q, k, sms, st);
}
