// ssa_mass.cu -- attention weight that each cached key received
// (ssa_attn_mass) on B200 (sm_100a).
//
// Given the rows' log-sum-exp, the weight of key j is a sum over query rows of
// exp(scale q.k_j - lse).  The scores are computed on tcgen05 and summed without
// atomics and without writing a probability anywhere.  Query rows are packed
// token-major over the G query heads of a key head (row i * G + g).
//
//   stream kernel: all G * window rows fit one operand (<= 256 rows).  S^T = K Q^T,
//     a thread a key, which adds its row's exponentials; the rows stay in
//     shared memory and the key tiles stream past, each read once: bound by
//     HBM (2 * d bytes a key and key head) up to about 64 rows, then by the
//     exponentials (16 a clock and SM).
//   prompt kernel: more rows.  Keys stay and the row tiles stream past from L2:
//     bound by the exponentials, 1,024 clocks a 128 x 128 tile against 512 for
//     its matrix product.
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
constexpr int NT = 640;  // warp 0 producer, 1 MMA, 2 rows and lse, 3 zero fill, 4-19 sums, in four groups
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

// -lse in log2 units; +inf, which only a lse of -inf gives, marks a row that has
// no keys or is not there: its exponentials do not count.  (NaN and +inf do.)
__device__ __forceinline__ float neg_lse2(const Params& p, int b, int hkv, int r) {
  const int i = p.Lq - p.W + r / p.G;
  if (i >= p.Lq) return INFINITY;
  return -p.lse[((size_t)b * p.Hq + hkv * p.G + r % p.G) * p.Lq + i] * LOG2E;
}

template <int NC>
__device__ __forceinline__ void load_columns(uint32_t taddr, float* x) {
  if constexpr (NC == 16) ssa::tmem_ld16f(taddr, x);
  else ssa::tmem_ld32f(taddr, x);
}

// Adds exp2(s c + nl) over NC columns.  MASK: columns below `first`, and rows without
// keys (nl = +inf), whose scores may be anything, do not count.
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
        p0 = i + 2 * h >= first && (h ? l.z : l.x) != INFINITY ? p0 : 0.f;
        p1 = i + 2 * h + 1 >= first && (h ? l.w : l.y) != INFINITY ? p1 : 0.f;
      }
      acc[h] = ssa::fadd2(acc[h], ssa::f2_pack(p0, p1));
    }
  }
}
// The same over NC columns of S^T at `at`, 32 (16) at a time; `after` runs once they are in registers.
template <int NC, class After>
__device__ __forceinline__ void add_tile(uint32_t at, const float* nl, float c, bool mask, int first, uint64_t (&acc)[2],
                                         After after) {
  constexpr int CH = NC < 32 ? NC : 32;
#pragma unroll
  for (int i = 0; i < NC; i += CH) {
    float x[CH];
    load_columns<CH>(at + i, x);
    ssa::tmem_wait_ld();
    if (i + CH == NC) after();
    if (mask) add_columns<CH, true>(x, nl + i, c, first - i, acc);
    else add_columns<CH, false>(x, nl + i, c, 0, acc);
  }
}
__device__ __forceinline__ float total(const uint64_t (&acc)[2]) {
  float a, b, c, d;
  ssa::f2_unpack(acc[0], a, b);
  ssa::f2_unpack(acc[1], c, d);
  return (a + b) + (c + d);
}

// ============================================================ stream kernel

template <int D, int N>
struct StreamSmem {
  static constexpr int NB = N <= 128 ? 4 : 2;  // S^T buffers; a group per tile, or two that halve its columns
  static constexpr int NC = N / (4 / NB);      // columns of a group
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
  constexpr int KST = L::KST, NB = L::NB, NC = L::NC;
  constexpr bool HALVES = NB == 2;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t kfull[KST], kempty[KST], q_full, q_empty, lse_full[2], lse_empty[2], s_full[NB], s_empty[NB], done;
  __shared__ uint64_t half_full[2], half_empty[2];
  __shared__ float half_sum[2][BK];
  __shared__ __align__(16) float nlse[2][N];
  __shared__ int bare[2];  // some column's row has no keys
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
      mbar_init(smem_u32(&lse_empty[i]), 16);
      mbar_init(smem_u32(&half_full[i]), 4);
      mbar_init(smem_u32(&half_empty[i]), 4);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), HALVES ? 8 : 4);
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
          if (!waits(&kfull[st], (g / KST) & 1) || !waits(&s_empty[g % NB], ((g / NB) & 1) ^ 1)) {
            ok = false;
            break;
          }
          ssa::tc_fence_after();
#pragma unroll
          for (int k16 = 0; k16 < D / 16; ++k16) {
            const uint32_t in = (k16 & 3) * 32;
            ssa::mma_ss_warp(leader, tmem + 512 / NB * (g % NB),
                        ssa::smem_desc_sw128(k_s + st * L::K_BYTES + (k16 >> 2) * BK * 128 + in, 16, 1024),
                        ssa::smem_desc_sw128(q_s + (k16 >> 2) * N * 128 + in, 16, 1024), idesc, k16 > 0);
          }
          ssa::mma_commit_warp(leader, smem_u32(&s_full[g % NB]));
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
      bool none = false;
#pragma unroll 1
      for (int r = lane; r < N; r += 32) {
        const float l = r < p.G * p.W ? neg_lse2(p, s.b, s.in, r) : INFINITY;
        none |= l == INFINITY;
        nlse[n & 1][r] = l;
      }
      none = __any_sync(0xffffffffu, none);
      if (lane == 0) bare[n & 1] = none;
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
    // group gr: tiles gr, gr + 4, ...; with halves tiles gr & 1, + 2, ..., columns of half gr >> 1
    const int gr = (warp - 4) >> 2, buf = gr % NB, half = HALVES ? gr >> 1 : 0;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 512 / NB * buf + NC * half;
    const int row = (warp & 3) * 32 + lane;
    int g = 0, n = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const int len = clamp_len(p.lens, s.b, p.cap);
      const size_t out = ((size_t)s.b * p.Hkv + s.in) * p.cap;
      ok = __all_sync(0xffffffffu, wait(&lse_full[n & 1], (n >> 1) & 1));
      for (int t = 0; ok && t < s.nt; ++t, ++g) {
        if (g % NB != buf) continue;
        const int j0 = (s.kt0 + t) * BK, j = j0 + row;
        const float before = half == 0 && p.mass_in != nullptr && j < len ? p.decay * p.mass_in[out + j] : 0.f;
        ok = __all_sync(0xffffffffu, wait(&s_full[buf], (g / NB) & 1));
        if (!ok) break;
        ssa::tc_fence_after();
        // row i of the window sits at i + len - W: key j counts from there on
        const bool mask = bare[n & 1] || (p.causal && j0 + BK - 1 > len - p.W);
        // (a distance below zero counts from row 0 on, and its product with G may not fit 32 bits)
        const int first = p.causal ? max(j - len + p.W, 0) * p.G - NC * half : 0;
        uint64_t acc[2] = {ssa::f2_pack(0.f, 0.f), ssa::f2_pack(0.f, 0.f)};
        add_tile<NC>(lanes, &nlse[n & 1][NC * half], p.c, mask, first, acc, [&] {
          ssa::tc_fence_before();  // S is in registers: the buffer is free
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_empty[buf]));
        });
        float sum = total(acc);
        if (HALVES) {  // the second half's sum goes to the first half's group
          const uint32_t parity = (g / NB) & 1;
          ok = __all_sync(0xffffffffu, half == 1 ? wait(&half_empty[buf], parity ^ 1) : wait(&half_full[buf], parity));
          if (!ok) break;
          if (half == 1) half_sum[buf][row] = sum;
          else sum += half_sum[buf][row];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(half == 1 ? &half_full[buf] : &half_empty[buf]));
        }
        if (half == 0 && j < p.cap) p.mass_out[out + j] = j < len ? before + sum : 0.f;
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
constexpr int KB = 256;   // keys of a block
constexpr int NTP = 576;  // warp 0 producer, 1 MMA, 2-17 sums (18 warps get the registers of 20: 96, with 24 bytes spilled)

template <int D>
struct PromptSmem {
  static constexpr uint32_t K_BYTES = KB * D * 2;
  static constexpr uint32_t Q_BYTES = BN * D * 2;
  static constexpr int QST = D == 128 ? 4 : 8;
  static constexpr uint32_t TOTAL = 1024 + K_BYTES + QST * Q_BYTES;
};

// Block (cluster rank r of S): 256 keys of one (sequence, key head) and the r-th
// S-th of the row tiles that see them; the parts are added through distributed
// shared memory in rank order.  S = Q K^T, a thread a row and 64 of the keys:
// its lse is one register and its 64 sums stay in registers over all row
// tiles, added over the threads once at the end.  (A thread a key, as in the
// stream kernel, reads a lse from shared memory for every exponential: 352 us
// against 340 at 8,192 rows and keys of 32 / 8 heads, d = 128; 344 since a lse of
// NaN is kept to the keys that its row sees.)  256 keys, because every row tile
// comes from L2, 32 KB in the 2,048 clocks of its exponentials.  Those take 78 % of
// all clocks; a quarter of them by a polynomial on the fp32 pipe changed nothing,
// so what is left lies between tiles and blocks.
template <int D>
__global__ void __launch_bounds__(NTP, 1)
    mass_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ Params p) {
  using L = PromptSmem<D>;
  constexpr int QST = L::QST;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t k_full, qfull[QST], qempty[QST], s_full[2], s_empty[2], done;
  __shared__ float quad_sum[4][KB], part[KB];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // low keys first: under a causal mask they are seen by the most rows
  const int item = blockIdx.x / S, pairs = p.B * p.Hkv;
  const int kt = item / pairs, pair = item % pairs;
  const int b = pair / p.Hkv, hkv = pair % p.Hkv;
  const int len = clamp_len(p.lens, b, p.cap);
  const int j0 = kt * KB;
  float* out = p.mass_out + (size_t)pair * p.cap;
  const float* in = p.mass_in != nullptr ? p.mass_in + (size_t)pair * p.cap : nullptr;
  if (j0 >= len) {  // the same for every block of the cluster
    if (rank == 0 && tid < KB && j0 + tid < p.cap) out[j0 + tid] = 0.f;
    return;
  }
  // first row tile that sees the block's first key, and this rank's range
  const int t_first = p.causal ? min(max((j0 - len + p.W) / p.tok, 0), p.tiles) : 0;
  const int nt = p.tiles - t_first;
  const int t0 = t_first + (int)((long long)nt * rank / S), t1 = t_first + (int)((long long)nt * (rank + 1) / S);
  const uint32_t k_s = smem_u32(base), q_s = k_s + L::K_BYTES;

  if (tid == 32) {
    ssa::tma_prefetch_desc(&tm_q);
    ssa::tma_prefetch_desc(&tm_k);
  }
  if (tid == 0) {
    mbar_init(smem_u32(&k_full), 1);
    mbar_init(smem_u32(&done), 1);
    for (int i = 0; i < QST; ++i) {
      mbar_init(smem_u32(&qfull[i]), 1);
      mbar_init(smem_u32(&qempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), 16);
    }
    abort_flag = 0;
    ssa::fence_mbar_init();
  }
  if (warp == 1) {
    ssa::tmem_alloc(smem_u32(&tmem_base), 512);
    ssa::tmem_relinquish();
  }
  ssa::tc_fence_before();
  __syncthreads();
  ssa::tc_fence_after();
  const uint32_t tmem = tmem_base;
  const ssa::Waiter wait{&abort_flag, p.status, p.wait_ns};

  if (warp == 0) {
    if (lane == 0 && t0 < t1) {
      mbar_arrive_expect_tx(smem_u32(&k_full), L::K_BYTES);
#pragma unroll
      for (int x = 0; x < KB / BK; ++x)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          ssa::tma_load_4d(k_s + (c * KB + x * BK) * 128, &tm_k, smem_u32(&k_full), c * 64, hkv, j0 + x * BK, b);
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
      constexpr uint32_t idesc = ssa::idesc_bf16_f32(BN, KB, false, false);
      const bool ok = waits(&k_full, 0);
      for (int g = 0; ok && g < t1 - t0; ++g) {
        const int st = g % QST;
        if (!waits(&qfull[st], (g / QST) & 1) || !waits(&s_empty[g & 1], ((g >> 1) & 1) ^ 1)) break;
        ssa::tc_fence_after();
#pragma unroll
        for (int k16 = 0; k16 < D / 16; ++k16)
          ssa::mma_ss_warp(leader, tmem + KB * (g & 1),
                           ssa::smem_desc_sw128(q_s + st * L::Q_BYTES + (k16 >> 2) * BN * 128 + (k16 & 3) * 32, 16, 1024),
                           ssa::smem_desc_sw128(k_s + (k16 >> 2) * KB * 128 + (k16 & 3) * 32, 16, 1024), idesc, k16 > 0);
        ssa::mma_commit_warp(leader, smem_u32(&s_full[g & 1]));
        ssa::mma_commit_warp(leader, smem_u32(&qempty[st]));
      }
      ssa::mma_commit_warp(leader, smem_u32(&done));
      ssa::mbar_wait(smem_u32(&done), 0, DRAIN_NS);
    }
  } else {
    const int slice = (warp - 2) >> 2, qd = warp & 3, row = qd * 32 + lane;
    const uint32_t at = tmem + ((uint32_t)(32 * qd) << 16) + 64 * slice;
    const int ti = row / p.G;  // the row's token in its tile (p.tok: none)
    const float* lse = p.lse + ((size_t)b * p.Hq + hkv * p.G + row % p.G) * p.Lq;
    // -inf for a row that is not there.  (Only the load, a tile ahead: arithmetic here would wait for it, 394 us
    // against 348 in a row of calls at the sizes above.)
    auto lse_of = [&](int g) {
      const int i = p.Lq - p.W + (t0 + g) * p.tok + ti;
      return g < t1 - t0 && ti < p.tok && i < p.Lq ? lse[i] : -INFINITY;
    };
    const uint64_t c2 = ssa::f2_pack(p.c, p.c);
    uint64_t acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = ssa::f2_pack(0.f, 0.f);
    float next = lse_of(0);
#pragma unroll 1
    for (int g = 0; g < t1 - t0; ++g) {
      const float nl = -next * LOG2E;  // +inf: a row that has no keys or is not there
      next = lse_of(g + 1);
      // keys of the slice that the row sees: the first `sees`; a row without keys none
      int sees = 64;
      if (p.causal) sees = min((t0 + g) * p.tok + ti + len - p.W - (j0 + 64 * slice) + 1, 64);
      if (nl == INFINITY) sees = 0;
      const bool mask = __any_sync(0xffffffffu, sees < 64);
      if (!__all_sync(0xffffffffu, wait(&s_full[g & 1], (g >> 1) & 1))) break;
      ssa::tc_fence_after();
      const uint64_t nl2 = ssa::f2_pack(nl, nl);
#pragma unroll
      for (int i = 0; i < 64; i += 16) {
        float x[16];
        ssa::tmem_ld16f(at + KB * (g & 1) + i, x);
        ssa::tmem_wait_ld();
        if (i == 48) {  // S is in registers: the buffer is free
          ssa::tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_empty[g & 1]));
        }
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          ssa::f2_unpack(ssa::ffma2(ssa::f2_pack(x[e], x[e + 1]), c2, nl2), x[e], x[e + 1]);
        if (mask) {  // (the whole exponent: a score or a lse may be NaN)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = i + e < sees ? x[e] : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          acc[(i + e) / 2] = ssa::fadd2(acc[(i + e) / 2], ssa::f2_pack(ex2(x[e]), ex2(x[e + 1])));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[32];
#pragma unroll
      for (int e = 0; e < 32; e += 2) ssa::f2_unpack(acc[16 * h + e / 2], y[e], y[e + 1]);
      quad_sum[qd][64 * slice + 32 * h + lane] = ssa::reduce_across<32>(y, [](float u, float v) { return u + v; });
    }
  }
  ssa::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ssa::tc_fence_after();
    ssa::tmem_dealloc(tmem, 512);
  }
  if (tid < KB) part[tid] = (quad_sum[0][tid] + quad_sum[1][tid]) + (quad_sum[2][tid] + quad_sum[3][tid]);
  if (S > 1) cluster.sync();
  if (rank == 0 && tid < KB && j0 + tid < p.cap) {
    float sum = 0.f;
    for (int r = 0; r < S; ++r) sum += *cluster.map_shared_rank(&part[tid], r);
    const int j = j0 + tid;
    out[j] = j < len ? (in != nullptr ? p.decay * in[j] + sum : sum) : 0.f;
  }
  if (S > 1) cluster.sync();  // rank 0 still reads the others' sums
}

template <class Kernel>
static int launch(Kernel* kernel, int threads, size_t smem, long long grid, int cluster, const CUtensorMap& q, const CUtensorMap& k,
                  const Params& p, cudaStream_t st) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SSA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
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
#define SSA_STREAM(N) launch(mass_stream_kernel<D, N>, NT, StreamSmem<D, N>::TOTAL, grid, 1, mq, mk, p, st)
    if (R <= 16) return SSA_STREAM(16);
    if (R <= 32) return SSA_STREAM(32);
    if (R <= 64) return SSA_STREAM(64);
    if (R <= 128) return SSA_STREAM(128);
    return SSA_STREAM(256);
#undef SSA_STREAM
  }
  if (!ssa::tma_map_bf16_box(&mq, q, p.B, p.Lq, p.Hq, D, p.G, p.tok)) return SSA_ERR_CUDA;
  // A cluster shares its keys' rows.  Under a causal mask a block's rows go from
  // all to none, and few large blocks would leave SMs idle at the end: two blocks
  // share while there are fewer than two an SM, and four or eight while that
  // still leaves fewer than two an SM, since clusters of four and eight leave SMs
  // of some GPCs unused.  Measured at d = 128, 4 query heads a key head, clusters
  // of 1, 2, 4, 8 (us), blocks before sharing: 16: 94 55 35 24; 48: 137 78 47 63;
  // 64: 97 58 46 67; 128: 185 106 127 168; 256: 358 343 406 510; 768: 2,699 2,703
  // 3,238 3,703.  Without the mask all blocks take the same time and what counts is
  // how they divide into rounds of the SMs, which this does not work out: shared
  // until there are two an SM (20: 218 119 68 74; 64: 98 59 66 94; 96: 141 148 126
  // 167; 160: 436 341 306 376).
  const long long items = pairs * ((p.cap + (long long)KB - 1) / KB);
  int cs = 1;
  while (cs < 8 && items * cs * (p.causal && cs > 1 ? 2 : 1) < 2 * sms && p.tiles >= cs * 4) cs *= 2;
  const long long grid = items * cs;
  if (grid > 0x7fffffff) return SSA_ERR_UNSUPPORTED;
  return launch(mass_prompt_kernel<D>, NTP, PromptSmem<D>::TOTAL, grid, cs, mq, mk, p, st);
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
  const size_t mass_bytes = (size_t)B * Hkv * cap * 4;
  const ssa::Span made{mass_out, mass_bytes};
  const ssa::Span in[5] = {{q, (size_t)B * Lq * Hq * d * 2}, {k, (size_t)B * cap * Hkv * d * 2}, {lse, (size_t)B * Hq * Lq * 4},
                           {lens, (size_t)B * 4}, {mass_in == mass_out ? nullptr : mass_in, mass_bytes}};
  for (const ssa::Span& x : in)
    if (ssa::overlap(made, x)) return SSA_ERR_INVALID_ARG;
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
