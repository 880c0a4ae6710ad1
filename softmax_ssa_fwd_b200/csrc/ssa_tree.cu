// ssa_tree.cu -- attention of drafted tokens (a tree, a chain, one token) over
// key/value caches of different lengths (ssa_decode_tree) on B200 (sm_100a).
//
// out_i = sum_j exp(s_ij - m) v_j / sum_j exp(s_ij - m), s = scale q.k, over the
// keys a row sees: the cache before the draft, and the draft keys of its mask.
// One pass over the keys with the running max m and sum of a softmax.
//
// Bound: K and V are read once for all G * T query rows that share a key head
// (4 * d bytes a key); a row costs 4 * d flops a key, so up to 256 rows the
// read takes longer than the tensor and exponential work.  The tiles of all
// sequences are spread evenly over the SMs (sched.cuh), whatever the lengths;
// where a (sequence, key head) lies in several blocks, each writes its
// unnormalised accumulator with (max, sum) and a second kernel, launched early
// and waiting on the first, merges them in block order.
//
// Query rows are packed token-major, row (i - first) * G + g.  Two kernels, by
// the rows R that share a key head; both have a warp that loads K and V, one
// that issues the products (tcgen05), one that loads Q, one that makes V safe
// and two softmax groups of four warps.
//   few rows (R <= 32): S^T = K Q^T and O^T += V^T P^T, a thread a key, so the
//     exponentials and the tensor work follow R (padded to 16 or 32) and not the
//     128 rows of an operand tile, and O is written with neighbouring columns
//     in neighbouring threads.  P goes through shared memory.
//   many rows: S = Q K^T and O += P V, a thread a row, P as bf16 in TMEM over
//     its S.  More than two 128-row tiles repeat the walk over the keys.
// Where a block has at most 128 rows the groups take alternate key tiles, one's
// products under the other's exponentials, each with its own accumulator,
// added at the end of a segment; with two row tiles each group has its own.
//
// Values that a row must not see: a hidden score becomes -inf, so P = 0; but
// 0 * inf and 0 * NaN are NaN, so one warp writes zeros over V rows past the last
// draft key, and over the non-finite elements of draft keys, which the epilogue
// adds to the rows that do see them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/ssa_cache.h"
#include "internal.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace ssa_tree {

using ssa::clamp_len;
using ssa::mbar_arrive;
using ssa::mbar_arrive_expect_tx;
using ssa::mbar_init;
using ssa::Seg;
using ssa::SegWalk;
using ssa::smem_u32;

constexpr int BK = 128;  // keys per tile
constexpr int BM = 128;  // rows per row tile (many rows)
constexpr int TMAX = 128;
constexpr int NT = 384;
constexpr int NBAD = 8;  // segments whose list of non-finite draft values is kept
constexpr unsigned long long DRAIN_NS = 2000000000ull;
constexpr float LN2 = 0.69314718055994531f;

struct Params {
  const __nv_bfloat16* v;
  __nv_bfloat16* out;
  float* lse;
  const int32_t* lens;
  const uint32_t* mask;
  float* o_part;    // [2 C, RT, d]: block c's first segment at 2 c, its last at 2 c + 1
  float2* ml_part;  // [2 C, RT]: max (log2 units), sum
  int4* segs;       // [B, Hkv * RG]: first block, its slot, last block
  int* status;
  unsigned long long wait_ns;
  int B, T, Hq, Hkv, G, cap, words;
  int tok, RG, RT;      // tokens per row tile, row groups, rows per group
  int C;                // blocks
  float c;              // scale * log2(e)
  bool stream_kv;       // the keys are read once
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// keys of sequence b with its draft, at least 1
__device__ __forceinline__ int key_count(const Params& p, int b) {
  return min(clamp_len(p.lens, b, p.cap) + p.T, p.cap);  // cap + T < 2^31
}
__device__ __forceinline__ int tile_count(const Params& p, int b) { return (key_count(p, b) + BK - 1) / BK; }

// Word w of a row's mask with the bits of draft keys that exist (t < tb).
__device__ __forceinline__ uint32_t mask_word(const uint32_t* row, int w, int tb) {
  const int left = tb - 32 * w;
  if (left <= 0) return 0u;
  return row[w] & (left >= 32 ? 0xffffffffu : (1u << left) - 1u);
}
// Bit e: the row sees the key at draft number t0 + e (negative: cached).
__device__ __forceinline__ uint32_t sees32(const uint32_t* row, int t0, int tb) {
  if (t0 + 31 < 0) return 0xffffffffu;
  if (t0 >= tb) return 0u;
  if (t0 < 0) return ((1u << -t0) - 1u) | (mask_word(row, 0, tb) << -t0);
  return __funnelshift_r(mask_word(row, t0 >> 5, tb), mask_word(row, (t0 >> 5) + 1, tb), t0 & 31);
}

// What the merge needs to know of a segment: where its parts are.
__device__ __forceinline__ void note_segment(const Params& p, const Seg& s, int n) {
  int* at = reinterpret_cast<int*>(p.segs + (size_t)s.b * (p.Hkv * p.RG) + s.in);
  if (s.kt0 == 0) {
    at[0] = blockIdx.x;
    at[1] = 2 * blockIdx.x + (n > 0 ? 1 : 0);
  }
  if (s.kt0 + s.nt == s.tiles) at[2] = blockIdx.x;
}

// One warp's pass over the V tiles of a block: those with keys that not every
// row sees are cleaned before the products read them.  (Element positions are
// swizzled within a row's 128-byte pieces; what is done here does not depend on
// them.)  bad: the draft keys of each segment that had non-finite values.
template <int D, int VST>
__device__ __forceinline__ void make_v_safe(const Params& p, SegWalk walk, const ssa::Waiter& wait, uint8_t* v_ring,
                                            const uint64_t* vfull, const uint64_t* vsafe,
                                            uint32_t (*bad)[TMAX / 32]) {
  constexpr uint32_t KV_BYTES = BK * D * 2;
  const int lane = threadIdx.x & 31;
  Seg s;
  int g = 0, n = 0;
  while (walk.next(s)) {
    const int len = clamp_len(p.lens, s.b, p.cap), keys = key_count(p, s.b);
    if (lane < TMAX / 32) bad[n % NBAD][lane] = 0u;
    __syncwarp();
    for (int t = 0; t < s.nt; ++t, ++g) {
      const int vs = g % VST, j0 = (s.kt0 + t) * BK;
      if (!__all_sync(0xffffffffu, wait(&vfull[vs], (g / VST) & 1))) return;
      if (j0 + BK > len) {
        uint8_t* tile = v_ring + vs * KV_BYTES;
        const int r0 = max(0, len - j0), r1 = min(BK, keys - j0);
        for (int e = r0 * 8 + lane; e < BK * 8; e += 32) {
          const int r = e >> 3;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint4* at = reinterpret_cast<uint4*>(tile + c * BK * 128) + e;
            if (r >= r1) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              uint4 x = *at;
              uint32_t* y = &x.x;
              bool hit = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((y[i] & 0x7f80u) == 0x7f80u) {
                  y[i] &= 0xffff0000u;
                  hit = true;
                }
                if ((y[i] & 0x7f800000u) == 0x7f800000u) {
                  y[i] &= 0x0000ffffu;
                  hit = true;
                }
              }
              if (hit) {
                *at = x;
                const int d = j0 + r - len;
                atomicOr(&bad[n % NBAD][d >> 5], 1u << (d & 31));
              }
            }
          }
        }
        ssa::fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&vsafe[vs]));
    }
    ++n;
  }
}

// One thread's loads of the K and V tiles of a block.
template <int D, int KST, int VST>
__device__ __forceinline__ void load_kv(const Params& p, SegWalk walk, const ssa::Waiter& wait, const CUtensorMap* tm_k,
                                        const CUtensorMap* tm_v, uint32_t k_s, uint32_t v_s, const uint64_t* kfull,
                                        const uint64_t* kempty, const uint64_t* vfull, const uint64_t* vempty) {
  constexpr uint32_t KV_BYTES = BK * D * 2;
  // read once: evict-first keeps the parts, which the merge reads, in L2
  const uint64_t policy = ssa::l2_evict_first_policy();
  auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int hkv, int j0, int b) {
    mbar_arrive_expect_tx(bar, KV_BYTES);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      if (p.stream_kv) ssa::tma_load_4d_hint(dst + c * BK * 128, map, bar, c * 64, hkv, j0, b, policy);
      else ssa::tma_load_4d(dst + c * BK * 128, map, bar, c * 64, hkv, j0, b);
    }
  };
  Seg s;
  int g = 0, kdone = 0, vdone = 0;
  bool ok = true;
  while (ok && walk.next(s))
    for (int t = 0; t < s.nt; ++t, ++g) {
      const int ks = g % KST, vs = g % VST, hkv = s.in / p.RG, j0 = (s.kt0 + t) * BK;
      ok = wait(&kempty[ks], ((g / KST) & 1) ^ 1);
      if (!ok) break;
      load(k_s + ks * KV_BYTES, tm_k, smem_u32(&kfull[ks]), hkv, j0, s.b);
      kdone = g + 1;
      ok = wait(&vempty[vs], ((g / VST) & 1) ^ 1);
      if (!ok) break;
      load(v_s + vs * KV_BYTES, tm_v, smem_u32(&vfull[vs]), hkv, j0, s.b);
      vdone = g + 1;
    }
  // nothing in flight when the block ends
  for (int t = max(0, kdone - KST); t < kdone; ++t) ssa::mbar_wait(smem_u32(&kfull[t % KST]), (t / KST) & 1, DRAIN_NS);
  for (int t = max(0, vdone - VST); t < vdone; ++t) ssa::mbar_wait(smem_u32(&vfull[t % VST]), (t / VST) & 1, DRAIN_NS);
}

// ============================================================ few rows

// N: rows, padded.
template <int D, int N>
struct FewSmem {
  static constexpr uint32_t Q_BYTES = N * D * 2;
  static constexpr uint32_t KV_BYTES = BK * D * 2;
  static constexpr uint32_t P_BYTES = N * BK * 2;
  // (d = 64: the V^T operand has 128 rows, of which the upper half, never used, are what follows the V tile in
  // shared memory: 16 KB have to)
  static constexpr uint32_t P_ALL = 2 * P_BYTES < 16384 ? 16384 : 2 * P_BYTES;
  static constexpr int FIT = (int)((215 * 1024 - Q_BYTES - P_ALL) / KV_BYTES);
  static constexpr int KST = (FIT + 1) / 2 < 4 ? (FIT + 1) / 2 : 4;
  static constexpr int VST = FIT / 2 < 4 ? FIT / 2 : 4;
  static constexpr uint32_t TOTAL = 1024 + Q_BYTES + (KST + VST) * KV_BYTES + P_ALL;
};

// Whether any of the 128 threads at named barrier `id` says so.
__device__ __forceinline__ bool any_of_group(uint32_t id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, float* x) {
  if constexpr (N == 16) ssa::tmem_ld16f(at, x);
  else ssa::tmem_ld32f(at, x);
}

template <int D, int N>
__global__ void __launch_bounds__(NT, 1)
    tree_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using L = FewSmem<D, N>;
  constexpr int KST = L::KST, VST = L::VST;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t kfull[KST], kempty[KST], vfull[VST], vempty[VST], vsafe[VST];
  __shared__ uint64_t q_full, q_empty, s_full[2], p_ready[2], pv_done[2], o_done, o_empty, done;
  __shared__ __align__(16) float neg_m[2][N], factor[2][N];   // -max * c, what the accumulators are multiplied by
  __shared__ float row_m[2][N], warp_top[2][4][N], warp_sum[2][2][4][N], seg_m[2][2][N];
  __shared__ __align__(16) float2 weight[2][N];
  __shared__ uint4 row_mask[2][N];
  __shared__ uint32_t bad[NBAD][TMAX / 32];
  __shared__ int pref[ssa::MAX_SEQS + 1];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_s = smem_u32(base), k_s = q_s + L::Q_BYTES, v_s = k_s + KST * L::KV_BYTES,
                 p_s = v_s + VST * L::KV_BYTES;

  if (tid == 32) {
    ssa::tma_prefetch_desc(&tm_q);
    ssa::tma_prefetch_desc(&tm_k);
    ssa::tma_prefetch_desc(&tm_v);
  }
  if (tid == 0) {
    for (int i = 0; i < KST; ++i) {
      mbar_init(smem_u32(&kfull[i]), 1);
      mbar_init(smem_u32(&kempty[i]), 1);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(smem_u32(&vfull[i]), 1);
      mbar_init(smem_u32(&vempty[i]), 1);
      mbar_init(smem_u32(&vsafe[i]), 1);
    }
    mbar_init(smem_u32(&q_full), 1);
    mbar_init(smem_u32(&q_empty), 1);
    mbar_init(smem_u32(&o_done), 1);
    mbar_init(smem_u32(&o_empty), 8);
    mbar_init(smem_u32(&done), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_ready[i]), 4);
      mbar_init(smem_u32(&pv_done[i]), 1);
    }
    abort_flag = 0;
    ssa::fence_mbar_init();
  }
  if (warp == 1) {
    ssa::tmem_alloc(smem_u32(&tmem_base), 512);
    ssa::tmem_relinquish();
  }
  if (warp == 2) ssa::tile_prefix(pref, p.B, [&](int b) { return tile_count(p, b); });
  if (p.RT < N) {  // rows of Q that are never loaded: zero
    for (int e = tid; e < (int)(L::Q_BYTES / 16); e += NT)
      reinterpret_cast<uint4*>(base)[e] = make_uint4(0u, 0u, 0u, 0u);
    ssa::fence_proxy_async_smem();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ssa::tc_fence_before();
  __syncthreads();
  ssa::tc_fence_after();
  const uint32_t tmem = tmem_base;
  const ssa::Waiter wait{&abort_flag, p.status, p.wait_ns};
  SegWalk walk(pref, p.B, p.Hkv, blockIdx.x, gridDim.x);
  Seg s;
  // S^T of tile g at column 128 * (g & 1), O^T of group w, which takes the tiles of g & 1 = w, at 256 + 128 * w

  if (warp == 0) {
    if (lane == 0) load_kv<D, KST, VST>(p, walk, wait, &tm_k, &tm_v, k_s, v_s, kfull, kempty, vfull, vempty);
  } else if (warp == 1) {
    {
      const uint32_t leader = ssa::elect_one();
      auto waits = [&](const uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
      constexpr uint32_t idesc_s = ssa::idesc_bf16_f32(BK, N, false, false);
      constexpr uint32_t idesc_o = ssa::idesc_bf16_f32(128, N, true, false);
      SegWalk walk_s = walk;
      Seg ss;
      int t_s = 0, n_s = 0, g_s = 0;
      bool more = walk_s.next(ss);
      auto issue_s = [&]() -> bool {
        const int ks = g_s % KST;
        if (t_s == 0 && !waits(&q_full, n_s & 1)) return false;
        if (!waits(&kfull[ks], (g_s / KST) & 1)) return false;
        ssa::tc_fence_after();
#pragma unroll
        for (int k16 = 0; k16 < D / 16; ++k16) {
          const uint32_t in = (k16 & 3) * 32;
          ssa::mma_ss_warp(leader, tmem + 128 * (g_s & 1),
                      ssa::smem_desc_sw128(k_s + ks * L::KV_BYTES + (k16 >> 2) * BK * 128 + in, 16, 1024),
                      ssa::smem_desc_sw128(q_s + (k16 >> 2) * N * 128 + in, 16, 1024), idesc_s, k16 > 0);
        }
        ssa::mma_commit_warp(leader, smem_u32(&s_full[g_s & 1]));
        ssa::mma_commit_warp(leader, smem_u32(&kempty[ks]));
        ++g_s;
        if (++t_s == ss.nt) {
          ssa::mma_commit_warp(leader, smem_u32(&q_empty));
          t_s = 0;
          ++n_s;
          more = walk_s.next(ss);
        }
        return true;
      };
      bool ok = true;
      for (int i = 0; i < 2 && ok && more; ++i) ok = issue_s();
      int g = 0, n = 0;
      while (ok && walk.next(s)) {
        uint32_t acc[2] = {0u, 0u};
        for (int t = 0; ok && t < s.nt; ++t, ++g) {
          const int w = g & 1, vs = g % VST, o = w;
          if (!waits(&p_ready[w], (g >> 1) & 1) || !waits(&vfull[vs], (g / VST) & 1) ||
              !waits(&vsafe[vs], (g / VST) & 1) || (t == 0 && !waits(&o_empty, (n & 1) ^ 1))) {
            ok = false;
            break;
          }
          ssa::tc_fence_after();
#pragma unroll
          for (int k16 = 0; k16 < BK / 16; ++k16) {
            ssa::mma_ss_warp(leader, tmem + 256 + 128 * o,
                        ssa::smem_desc_sw128(v_s + vs * L::KV_BYTES + k16 * 16 * 128, BK * 128, 1024),
                        ssa::smem_desc_sw128(p_s + o * L::P_BYTES + (k16 >> 2) * N * 128 + (k16 & 3) * 32, 16, 1024),
                        idesc_o, acc[o]);
            acc[o] = 1u;
          }
          ssa::mma_commit_warp(leader, smem_u32(&vempty[vs]));
          ssa::mma_commit_warp(leader, smem_u32(&pv_done[o]));
          if (t == s.nt - 1) ssa::mma_commit_warp(leader, smem_u32(&o_done));
          if (more) ok = issue_s();  // over the S of tile g, which the softmax has read
        }
        ++n;
      }
      ssa::mma_commit_warp(leader, smem_u32(&done));
      ssa::mbar_wait(smem_u32(&done), 0, DRAIN_NS);  // no MMA in flight when TMEM is freed
    }
  } else if (warp == 2) {
    if (lane == 0) {
      int n = 0;
      while (walk.next(s)) {
        note_segment(p, s, n);
        if (!wait(&q_empty, (n & 1) ^ 1)) break;
        mbar_arrive_expect_tx(smem_u32(&q_full), (uint32_t)(p.RT * D * 2));
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          ssa::tma_load_4d(q_s + c * N * 128, &tm_q, smem_u32(&q_full), c * 64, s.in * p.G, 0, s.b);
        ++n;
      }
      if (n > 0) ssa::mbar_wait(smem_u32(&q_full), (n - 1) & 1, DRAIN_NS);
    }
  } else if (warp == 3) {
    make_v_safe<D, VST>(p, walk, wait, base + L::Q_BYTES + KST * L::KV_BYTES, vfull, vsafe, bad);
  } else {
    // The group's four warps meet at named barriers, so none of them leaves
    // before the walk is over: a wait that gave up lets the others give up at
    // once, and what is computed from then on is not used.
    const int wg = (warp - 4) >> 2, qd = warp & 3, key = qd * 32 + lane, gt = tid & 127;
    const uint32_t bar = 1 + wg;
    const uint32_t lanes = tmem + ((uint32_t)(32 * qd) << 16);
    const float c = p.c;
    const uint64_t c2 = ssa::f2_pack(c, c);
    // P[row][key], K-major in 128-byte-swizzled boxes of 64 keys.  Neighbouring threads swap, so that each stores
    // two keys of a row: the even one of row r, the odd one of row r + 4, whose 16-byte pieces lie in the other
    // banks.  p_at: r = 0..3 of eight rows.
    uint32_t p_at[4];
    const uint32_t odd = lane & 1, p_pick = odd ? 0x3276u : 0x5410u;
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      const uint32_t r = e + 4 * odd;
      p_at[e] = p_s + wg * L::P_BYTES + (key >> 6) * (N * 128) + r * 128 + ((((key & 63) >> 3) ^ r) << 4) + (key & 6) * 2;
    }
    int g = 0, n = 0;
    uint32_t mine = 0;  // this group's tiles so far
    while (walk.next(s)) {
      const int len = clamp_len(p.lens, s.b, p.cap), tb = min(p.T, p.cap - len);
      if (gt < N) {
        uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);  // (a row that is not there sees everything: zeros)
        if (gt < p.RT) {
          const uint32_t* row = p.mask + ((size_t)s.b * p.T + gt / p.G) * p.words;
          m = make_uint4(mask_word(row, 0, tb), mask_word(row, 1, tb), mask_word(row, 2, tb), mask_word(row, 3, tb));
        }
        row_mask[wg][gt] = m;
      }
      uint64_t l[N / 2];  // this thread's part of the rows' sums
#pragma unroll
      for (int r = 0; r < N / 2; ++r) l[r] = ssa::f2_pack(0.f, 0.f);
      bool any = false, force = true;  // force: a row has no max yet
      const int t_first = (g ^ wg) & 1;
#pragma unroll 1
      for (int t = t_first; t < s.nt; t += 2) {
        const int gg = g + t;
        wait(&s_full[wg], (gg >> 1) & 1);
        __syncwarp();
        ssa::tc_fence_after();
        const int j = (s.kt0 + t) * BK + key - len;  // draft number of this thread's key, negative: cached
        const bool tail = (s.kt0 + t) * BK + BK > len;
        if (tail && !any) any_of_group(bar, false);  // the masks are in shared memory
        // x: the scores, then the exponents under the max in use.  The max only follows when a key is more
        // than 2^8 ahead (or a row has none yet): P stays below 2^8 and the sums in fp32, and the accumulators
        // are rarely rescaled.  Any row may send the group to FIND, but each row's max follows its own keys
        // alone: its bits do not depend on what other rows see.
        float x[N];
        enum { CHECK, FIND, APPLY } step = force ? FIND : CHECK;
#pragma unroll 1
        for (;;) {
          tmem_ld<N>(lanes + 128 * wg, x);
          ssa::tmem_wait_ld();
          if (tail && j >= 0) {
#pragma unroll
            for (int r = 0; r < N; ++r) {
              const uint32_t m = j < tb ? reinterpret_cast<const uint32_t*>(&row_mask[wg][r])[j >> 5] : 0u;
              x[r] = (m >> (j & 31)) & 1u ? x[r] : -INFINITY;
            }
          }
          if (step == FIND) {  // (uses x up: it is read again)
            const float top = ssa::reduce_across<N>(x, [](float u, float v) { return fmaxf(u, v); });
            if (lane < N) warp_top[wg][qd][lane] = top;
            any_of_group(bar, false);
            bool empty = false;
            if (gt < N) {
              const float old = any ? row_m[wg][gt] : -INFINITY;
              const float best = fmaxf(fmaxf(warp_top[wg][0][gt], warp_top[wg][1][gt]),
                                       fmaxf(warp_top[wg][2][gt], warp_top[wg][3][gt]));
              // (CHECK's own arithmetic, so that this row moves here iff it would have asked for it)
              const bool up = old == -INFINITY || fmaf(best, c, neg_m[wg][gt]) > 8.f;
              const float m = up ? fmaxf(best, old) : old;
              row_m[wg][gt] = m;
              empty = m == -INFINITY;
              neg_m[wg][gt] = empty ? 0.f : -m * c;
              factor[wg][gt] = old == -INFINITY ? 0.f : ex2((old - m) * c);
            }
            force = any_of_group(bar, empty);
            step = APPLY;
            continue;
          }
          float top = -INFINITY;
#pragma unroll
          for (int r = 0; r < N; r += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&neg_m[wg][r]);
            ssa::f2_unpack(ssa::ffma2(ssa::f2_pack(x[r], x[r + 1]), c2, ssa::f2_pack(m.x, m.y)), x[r], x[r + 1]);
            ssa::f2_unpack(ssa::ffma2(ssa::f2_pack(x[r + 2], x[r + 3]), c2, ssa::f2_pack(m.z, m.w)), x[r + 2],
                           x[r + 3]);
            top = ssa::fmax3(top, fmaxf(x[r], x[r + 1]), fmaxf(x[r + 2], x[r + 3]));
          }
          if (step == APPLY) {
            if (any) {
              wait(&pv_done[wg], (mine - 1) & 1);
              __syncwarp();
              ssa::tc_fence_after();
              const uint32_t o_col = lanes + 256 + 128 * wg;
#pragma unroll
              for (int r0 = 0; r0 < N; r0 += 16) {
                uint32_t u[16];
                float o[16];
                ssa::tmem_ld16f(o_col + r0, o);
                ssa::tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                  const float2 f = *reinterpret_cast<const float2*>(&factor[wg][r0 + r]);
                  u[r] = __float_as_uint(o[r] * f.x);
                  u[r + 1] = __float_as_uint(o[r + 1] * f.y);
                  l[(r0 + r) / 2] = ssa::fmul2(l[(r0 + r) / 2], ssa::f2_pack(f.x, f.y));
                }
                ssa::tmem_st16(o_col + r0, u);
              }
              ssa::tmem_wait_st();
            }
            break;
          }
          if (!any_of_group(bar, top > 8.f)) break;
          step = FIND;
        }
#pragma unroll
        for (int r = 0; r < N; r += 2) {
          x[r] = ex2(x[r]);
          x[r + 1] = ex2(x[r + 1]);
          l[r / 2] = ssa::fadd2(l[r / 2], ssa::f2_pack(x[r], x[r + 1]));
        }
        if (any) {  // the P V before this tile (a segment's first one follows a complete O)
          wait(&pv_done[wg], (mine - 1) & 1);
          __syncwarp();
        }
#pragma unroll
        for (int r8 = 0; r8 < N; r8 += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // rounded to bf16 for the tensor cores; the sums take the unrounded ones
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[r8 + e], x[r8 + e + 4]);
            const uint32_t u = *reinterpret_cast<const uint32_t*>(&b2);
            ssa::st_shared_u32(p_at[e] + r8 * 128, __byte_perm(u, __shfl_xor_sync(0xffffffffu, u, 1), p_pick));
          }
        }
        ssa::fence_proxy_async_smem();
        ssa::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_ready[wg]));
        ++mine;
        any = true;
      }
      g += s.nt;

      // ---- end of the segment: the rows' sums over the group's threads
      float (*sums)[4][N] = warp_sum[n & 1];
      float y[N];
#pragma unroll
      for (int r = 0; r < N; r += 2) ssa::f2_unpack(l[r / 2], y[r], y[r + 1]);
      const float part_sum = ssa::reduce_across<N>(y, [](float u, float v) { return u + v; });
      if (lane < N) sums[wg][qd][lane] = part_sum;
      if (gt < N) seg_m[n & 1][wg][gt] = any ? row_m[wg][gt] : -INFINITY;
      ssa::named_bar_sync(3, 256);
      const bool whole = s.nt == s.tiles;
      const int slot = 2 * blockIdx.x + (n > 0 ? 1 : 0);  // a part is a block's first or its last segment
      if (gt < N) {
        const float m0 = seg_m[n & 1][0][gt], m1 = seg_m[n & 1][1][gt], m = fmaxf(m0, m1);
        float w0 = m0 == -INFINITY ? 0.f : ex2((m0 - m) * c), w1 = m1 == -INFINITY ? 0.f : ex2((m1 - m) * c);
        const float sum = fmaf((sums[0][0][gt] + sums[0][1][gt]) + (sums[0][2][gt] + sums[0][3][gt]), w0,
                               ((sums[1][0][gt] + sums[1][1][gt]) + (sums[1][2][gt] + sums[1][3][gt])) * w1);
        if (whole) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          w0 *= inv;
          w1 *= inv;
        }
        weight[wg][gt] = make_float2(w0, w1);
        if (gt < p.RT && wg == 0) {
          if (whole)
            p.lse[((size_t)s.b * p.Hq + s.in * p.G + gt % p.G) * p.T + gt / p.G] =
                sum == 0.f ? -INFINITY : (m * c + log2f(sum)) * LN2;
          else p.ml_part[(size_t)slot * p.RT + gt] = make_float2(m * c, sum);
        }
      }
      any_of_group(bar, false);
      wait(&o_done, n & 1);
      __syncwarp();
      ssa::tc_fence_after();
      // this thread: column `key` of the head, of half of the rows
      const uint32_t* bd = bad[n % NBAD];
      const bool fix = (bd[0] | bd[1] | bd[2] | bd[3]) != 0u;
      constexpr int CH = N / 2;
      const int r0 = wg * CH;
      // (of a segment of one tile only one group has an accumulator)
      const bool has0 = s.nt > 1 || ((g - 1) & 1) == 0, has1 = s.nt > 1 || ((g - 1) & 1) == 1;
      float o[16], z[16];
      if (has0) ssa::tmem_ld16f(lanes + 256 + r0, o);
      if (has1) ssa::tmem_ld16f(lanes + 256 + 128 + r0, z);
      ssa::tmem_wait_ld();
      // O is in registers: the next segment may overwrite it
      ssa::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&o_empty));
      if (key < D) {
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          const float2 w = weight[wg][r0 + e];
          o[e] = (has0 ? o[e] * w.x : 0.f) + (has1 ? z[e] * w.y : 0.f);
        }
        if (fix) {
#pragma unroll 1
          for (int t = 0; t < tb; ++t) {
            if (!((bd[t >> 5] >> (t & 31)) & 1u)) continue;
            const float v = __bfloat162float(p.v[(((size_t)s.b * p.cap + len + t) * p.Hkv + s.in) * D + key]);
            if (isfinite(v)) continue;
#pragma unroll
            for (int e = 0; e < CH; ++e)
              if ((reinterpret_cast<const uint32_t*>(&row_mask[wg][r0 + e])[t >> 5] >> (t & 31)) & 1u) o[e] += v;
          }
        }
        const int left = p.RT - r0;
        if (!whole) {
          float* dst = p.o_part + ((size_t)slot * p.RT + r0) * D + key;
#pragma unroll
          for (int e = 0; e < CH; ++e)
            if (e < left) dst[e * D] = o[e];
        } else {
          int i = r0 / p.G, gq = r0 % p.G;
#pragma unroll
          for (int e = 0; e < CH; ++e) {
            if (e < left)
              p.out[(((size_t)s.b * p.T + i) * p.Hq + s.in * p.G + gq) * D + key] = __float2bfloat16_rn(o[e]);
            if (++gq == p.G) {
              gq = 0;
              ++i;
            }
          }
        }
      }
      any_of_group(bar, false);  // the masks and weights have been read
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

// ============================================================ many rows

// NQ: row tiles of a block.  1: the groups take alternate key tiles of the same
// rows; 2: each has its own rows and takes every key tile.
template <int D, int NQ>
struct ManySmem {
  static constexpr uint32_t Q_BYTES = BM * D * 2;  // a row tile
  static constexpr uint32_t KV_BYTES = BK * D * 2;
  static constexpr int PITCH = 20;  // floats a row of a warp's 32 x 16 output stage: no bank conflicts
  static constexpr uint32_t STAGE = 8 * 32 * PITCH * 4;
  static constexpr int FIT = (int)((212 * 1024 - NQ * Q_BYTES - STAGE) / KV_BYTES);  // K and V tiles
  static constexpr int KST = (FIT + 1) / 2 < 4 ? (FIT + 1) / 2 : 4;
  static constexpr int VST = FIT / 2 < 4 ? FIT / 2 : 4;
  static constexpr uint32_t TOTAL = 1024 + NQ * Q_BYTES + (KST + VST) * KV_BYTES + STAGE;
};

template <int D, int NQ>
__global__ void __launch_bounds__(NT, 1)
    tree_many_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using L = ManySmem<D, NQ>;
  constexpr int KST = L::KST, VST = L::VST;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t kfull[KST], kempty[KST], vfull[VST], vempty[VST], vsafe[VST];
  __shared__ uint64_t q_full, q_empty, s_full[2], p_ready[2], o_done, o_empty, ml_full[2], done;
  __shared__ float2 ml[2][2][NQ == 1 ? BM : 1];
  __shared__ uint32_t bad[NBAD][TMAX / 32];
  __shared__ int pref[ssa::MAX_SEQS + 1];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_s = smem_u32(base), k_s = q_s + NQ * L::Q_BYTES, v_s = k_s + KST * L::KV_BYTES;
  float* stage_all = reinterpret_cast<float*>(base + NQ * L::Q_BYTES + (KST + VST) * L::KV_BYTES);

  if (tid == 32) {
    ssa::tma_prefetch_desc(&tm_q);
    ssa::tma_prefetch_desc(&tm_k);
    ssa::tma_prefetch_desc(&tm_v);
  }
  if (tid == 0) {
    for (int i = 0; i < KST; ++i) {
      mbar_init(smem_u32(&kfull[i]), 1);
      mbar_init(smem_u32(&kempty[i]), 1);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(smem_u32(&vfull[i]), 1);
      mbar_init(smem_u32(&vempty[i]), 1);
      mbar_init(smem_u32(&vsafe[i]), 1);
    }
    mbar_init(smem_u32(&q_full), 1);
    mbar_init(smem_u32(&q_empty), 1);
    mbar_init(smem_u32(&o_done), 1);
    mbar_init(smem_u32(&o_empty), 8);
    mbar_init(smem_u32(&done), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_ready[i]), 4);
      mbar_init(smem_u32(&ml_full[i]), 8);
    }
    abort_flag = 0;
    ssa::fence_mbar_init();
  }
  if (warp == 1) {
    ssa::tmem_alloc(smem_u32(&tmem_base), 512);
    ssa::tmem_relinquish();
  }
  if (warp == 2) ssa::tile_prefix(pref, p.B, [&](int b) { return tile_count(p, b); });
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ssa::tc_fence_before();
  __syncthreads();
  ssa::tc_fence_after();
  const uint32_t tmem = tmem_base;
  const ssa::Waiter wait{&abort_flag, p.status, p.wait_ns};
  SegWalk walk(pref, p.B, p.Hkv * p.RG, blockIdx.x, gridDim.x);
  Seg s;

  if (warp == 0) {
    if (lane == 0) load_kv<D, KST, VST>(p, walk, wait, &tm_k, &tm_v, k_s, v_s, kfull, kempty, vfull, vempty);
  } else if (warp == 1) {
    {
      const uint32_t leader = ssa::elect_one();
      auto waits = [&](const uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
      constexpr uint32_t idesc_qk = ssa::idesc_bf16_f32(BM, BK, false, false);
      constexpr uint32_t idesc_pv = ssa::idesc_bf16_f32(BM, D, false, true);
      // Steps: softmax group h & 1 takes step h; a key tile is NQ steps.  S of
      // step h + 2 is issued after the P V of step h, whose P it overwrites.
      SegWalk walk_s = walk;
      Seg ss;
      int t_s = 0, n_s = 0, h_s = 0;
      bool more = walk_s.next(ss);
      auto issue_s = [&]() -> bool {
        const int w = h_s & 1, g = h_s / NQ, ks = g % KST;
        if (t_s == 0 && !waits(&q_full, n_s & 1)) return false;
        if (!waits(&kfull[ks], (g / KST) & 1)) return false;
        ssa::tc_fence_after();
#pragma unroll
        for (int k16 = 0; k16 < D / 16; ++k16) {
          const uint32_t o = (k16 >> 2) * (128 * 128) + (k16 & 3) * 32;
          ssa::mma_ss_warp(leader, tmem + 256 * w, ssa::smem_desc_sw128(q_s + (NQ == 2 ? w : 0) * L::Q_BYTES + o, 16, 1024),
                      ssa::smem_desc_sw128(k_s + ks * L::KV_BYTES + o, 16, 1024), idesc_qk, k16 > 0);
        }
        ssa::mma_commit_warp(leader, smem_u32(&s_full[w]));
        if (NQ == 1 || w == 1) ssa::mma_commit_warp(leader, smem_u32(&kempty[ks]));
        ++h_s;
        if (++t_s == ss.nt * NQ) {
          ssa::mma_commit_warp(leader, smem_u32(&q_empty));
          t_s = 0;
          ++n_s;
          more = walk_s.next(ss);
        }
        return true;
      };
      bool ok = true;
      for (int i = 0; i < 2 && ok && more; ++i) ok = issue_s();
      int h = 0, n = 0;
      while (ok && walk.next(s)) {
        uint32_t acc[2] = {0u, 0u};
        for (int t = 0; ok && t < s.nt * NQ; ++t, ++h) {
          const int w = h & 1, g = h / NQ, vs = g % VST;
          if (!waits(&p_ready[w], (h >> 1) & 1) || !waits(&vfull[vs], (g / VST) & 1) ||
              !waits(&vsafe[vs], (g / VST) & 1) || (t == 0 && !waits(&o_empty, (n & 1) ^ 1))) {
            ok = false;
            break;
          }
          ssa::tc_fence_after();
#pragma unroll
          for (int k16 = 0; k16 < BK / 16; ++k16) {
            ssa::mma_ts_warp(leader, tmem + 256 * w + 128, tmem + 256 * w + k16 * 8,
                        ssa::smem_desc_sw128(v_s + vs * L::KV_BYTES + k16 * 16 * 128, BK * 128, 1024), idesc_pv, acc[w]);
            acc[w] = 1u;
          }
          if (NQ == 1 || w == 1) ssa::mma_commit_warp(leader, smem_u32(&vempty[vs]));
          if (t == s.nt * NQ - 1) ssa::mma_commit_warp(leader, smem_u32(&o_done));
          if (more) ok = issue_s();
        }
        ++n;
      }
      ssa::mma_commit_warp(leader, smem_u32(&done));
      ssa::mbar_wait(smem_u32(&done), 0, DRAIN_NS);  // no MMA in flight when TMEM is freed
    }
  } else if (warp == 2) {
    if (lane == 0) {
      int n = 0;
      while (walk.next(s)) {
        note_segment(p, s, n);
        if (!wait(&q_empty, (n & 1) ^ 1)) break;
        mbar_arrive_expect_tx(smem_u32(&q_full), (uint32_t)(NQ * p.G * p.tok * D * 2));
        const int hq = s.in / p.RG * p.G, i0 = s.in % p.RG * (NQ * p.tok);
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            ssa::tma_load_4d(q_s + x * L::Q_BYTES + c * BM * 128, &tm_q, smem_u32(&q_full), c * 64, hq,
                             i0 + x * p.tok, s.b);
        ++n;
      }
      if (n > 0) ssa::mbar_wait(smem_u32(&q_full), (n - 1) & 1, DRAIN_NS);
    }
  } else if (warp == 3) {
    make_v_safe<D, VST>(p, walk, wait, base + NQ * L::Q_BYTES + KST * L::KV_BYTES, vfull, vsafe, bad);
  } else {
    const int wg = (warp - 4) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = lanes + 256 * wg, o_col = s_col + 128;
    const int row = (warp & 3) * 32 + lane, rows = p.tok * p.G;
    const float c = p.c;
    const uint64_t c2 = ssa::f2_pack(c, c);
    float* stage = stage_all + (warp - 4) * 32 * L::PITCH;
    int n = 0, g = 0;
    uint32_t cnt = 0;  // S tiles of this group so far
    bool ok = true;
    while (ok && walk.next(s)) {
      const int len = clamp_len(p.lens, s.b, p.cap), tb = min(p.T, p.cap - len);
      const int hkv = s.in / p.RG, i0 = s.in % p.RG * (NQ * p.tok) + (NQ == 2 ? wg : 0) * p.tok;  // the row tile's first token
      const int i = i0 + row / p.G;
      const bool valid = row < rows && i < p.T;
      const uint32_t* mrow = p.mask + ((size_t)s.b * p.T + (valid ? i : 0)) * p.words;
      float m = -INFINITY, l = 0.f;  // max in use (of q.k), sum
      const int t_first = NQ == 1 ? (g ^ wg) & 1 : 0;
#pragma unroll 1
      for (int t = t_first; t < s.nt; t += NQ == 1 ? 2 : 1) {
        ok = __all_sync(0xffffffffu, wait(&s_full[wg], cnt & 1));
        if (!ok) break;
        ++cnt;
        ssa::tc_fence_after();
        const int j0 = (s.kt0 + t) * BK;
        const bool mask = j0 + BK > len;
        // 64 columns at a time, read twice: a whole row does not fit the registers beside what else is held
        auto load = [&](int h, float* x) {
          ssa::tmem_ld64f(s_col + 64 * h, x);
          ssa::tmem_wait_ld();
          if (mask) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t see = valid ? sees32(mrow, j0 + 64 * h + 32 * w - len, tb) : 0u;
#pragma unroll
              for (int e = 0; e < 32; ++e) x[32 * w + e] = (see >> e) & 1u ? x[32 * w + e] : -INFINITY;
            }
          }
        };
        float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[64];
          load(h, x);
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            a0 = ssa::fmax3(a0, x[e], x[e + 1]);
            a1 = ssa::fmax3(a1, x[e + 2], x[e + 3]);
          }
        }
        const float tmax = fmaxf(a0, a1);
        // The max in use only follows when it is more than 2^8 behind: P stays
        // below 2^8 and the sums in fp32, and O is rarely rescaled.  Each row's
        // follows its own keys alone; operand rows that are not query rows hold
        // what was in shared memory and do not vote.
        const bool up = tmax * c > m * c + 8.f;
        if (t == t_first) {
          m = tmax;
        } else if (__any_sync(0xffffffffu, valid && up)) {
          // (S of this tile is complete, so the P V before it is too)
          const float f = up ? ex2((m - tmax) * c) : 1.f;
          m = up ? tmax : m;
          l *= f;
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            ssa::tmem_ld32(o_col + 32 * cc, o);
            ssa::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            ssa::tmem_st32(o_col + 32 * cc, o);
          }
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        const uint64_t mc2 = ssa::f2_pack(-mc, -mc);
        uint64_t sum[2] = {ssa::f2_pack(0.f, 0.f), ssa::f2_pack(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[64];
          load(h, x);
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float p0, p1;
            ssa::f2_unpack(ssa::ffma2(ssa::f2_pack(x[2 * e], x[2 * e + 1]), c2, mc2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum[e & 1] = ssa::fadd2(sum[e & 1], ssa::f2_pack(p0, p1));
            // rounded to bf16 for the tensor cores; the sum takes the unrounded ones
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
            pk[e] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          ssa::tmem_st32(s_col + 32 * h, pk);  // over columns that have been read
        }
        float s0, s1, s2, s3;
        ssa::f2_unpack(sum[0], s0, s1);
        ssa::f2_unpack(sum[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        ssa::tmem_wait_st();
        ssa::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_ready[wg]));
      }
      if (!ok) break;

      // ---- end of the segment
      const bool any = t_first < s.nt, other = NQ == 1 && (s.nt > 1 || !any);
      g += s.nt;
      float w0 = 1.f, w1 = 0.f;  // weights of this group's accumulator and of the other's
      if (NQ == 1) {
        ml[n & 1][wg][row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ml_full[n & 1]));
        ok = __all_sync(0xffffffffu, wait(&ml_full[n & 1], (n >> 1) & 1));
        if (!ok) break;
        const float2 y = ml[n & 1][wg ^ 1][row];
        const float M = fmaxf(m, y.x);
        w0 = m == -INFINITY ? 0.f : ex2((m - M) * c);
        w1 = y.x == -INFINITY ? 0.f : ex2((y.x - M) * c);
        m = M;
        l = wg == 0 ? fmaf(l, w0, y.y * w1) : fmaf(y.y, w1, l * w0);  // the same sum in both, to the bit
      }
      ok = __all_sync(0xffffffffu, wait(&o_done, n & 1));
      if (!ok) break;
      ssa::tc_fence_after();
      const bool whole = s.nt == s.tiles;
      const int slot = 2 * blockIdx.x + (n > 0 ? 1 : 0);  // a part is a block's first or its last segment
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        w0 *= inv;
        w1 *= inv;
      }
      const uint32_t* bd = bad[n % NBAD];
      const bool fix = (bd[0] | bd[1] | bd[2] | bd[3]) != 0u;
      // A row lies in one thread; through shared memory, 16 columns at a time, four
      // neighbouring threads write a row: this thread rows 8 e + lane / 4.
      int64_t dst[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = (warp & 3) * 32 + 8 * e + lane / 4, ri = i0 + r / p.G;
        dst[e] = r >= rows || ri >= p.T ? -1
                 : whole ? (((int64_t)s.b * p.T + ri) * p.Hq + hkv * p.G + r % p.G) * D
                         : ((int64_t)slot * p.RT + (NQ == 2 ? wg : 0) * rows + r) * D;
      }
      constexpr int COLS = NQ == 1 ? D / 2 : D;  // one row tile: each group writes half of the columns
      const int col0 = NQ == 1 ? wg * COLS : 0;
#pragma unroll 1
      for (int col = col0; col < col0 + COLS; col += 16) {
        float o[16], y[16];
        if (any) ssa::tmem_ld16f(o_col + col, o);
        if (other) ssa::tmem_ld16f(lanes + 256 * (wg ^ 1) + 128 + col, y);
        ssa::tmem_wait_ld();
        if (col + 16 >= col0 + COLS) {  // O is in registers: the next segment may overwrite it
          ssa::tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&o_empty));
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = (any ? o[e] * w0 : 0.f) + (other ? y[e] * w1 : 0.f);
        if (fix && valid) {
#pragma unroll 1
          for (int t = 0; t < tb; ++t) {
            if (!((bd[t >> 5] & mask_word(mrow, t >> 5, tb)) >> (t & 31) & 1u)) continue;
            const __nv_bfloat16* v = p.v + (((size_t)s.b * p.cap + len + t) * p.Hkv + hkv) * D + col;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float y = __bfloat162float(v[e]);
              if (!isfinite(y)) o[e] += y;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<float4*>(stage + lane * L::PITCH + 4 * e) =
              make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 y = *reinterpret_cast<const float4*>(stage + (8 * e + lane / 4) * L::PITCH + 4 * (lane & 3));
          if (dst[e] < 0) continue;
          const int64_t at = dst[e] + col + 4 * (lane & 3);
          if (whole) {
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(y.x, y.y), b1 = __floats2bfloat162_rn(y.z, y.w);
            *reinterpret_cast<uint2*>(p.out + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
          } else {
            *reinterpret_cast<float4*>(p.o_part + at) = y;
          }
        }
        __syncwarp();
      }
      if (valid && (NQ == 2 || wg == 0)) {
        if (whole)
          p.lse[((size_t)s.b * p.Hq + hkv * p.G + row % p.G) * p.T + i] =
              l == 0.f ? -INFINITY : (m * c + log2f(l)) * LN2;
        else p.ml_part[(size_t)slot * p.RT + (NQ == 2 ? wg : 0) * rows + row] = make_float2(m * c, l);
      }
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

// ============================================================ merge

// The parts of a query row's (sequence, key head, row group), in block order.
// WIDE: a block a row, every eighth part by a warp: for long caches of few
// heads, whose segments lie in many blocks.  Otherwise a warp a row.
constexpr int MW = 8;  // warps per block

template <int D, bool WIDE>
__global__ void __launch_bounds__(32 * MW) tree_merge_kernel(const __grid_constant__ Params p, int tokens) {
  constexpr int E = D / 32, STEP = WIDE ? MW : 1;
  __shared__ float acc[WIDE ? MW : 1][D];
  __shared__ float tot[MW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = WIDE ? blockIdx.x : blockIdx.x * MW + warp;
  const bool live = row < p.B * p.T * p.Hq;
  const int hq = row % p.Hq, bi = row / p.Hq, i = bi % p.T, b = live ? bi / p.T : 0;
  const int rg = i / tokens, in = hq / p.G * p.RG + rg;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // by every block: what follows in the stream needs both kernels
  if (!live) return;
  const int4 seg = p.segs[(size_t)b * (p.Hkv * p.RG) + in];
  // (after a wait that gave up the table may hold anything)
  const int c0 = max(seg.x, 0), c1 = min(seg.z, p.C - 1), first = min(max(seg.y, 0), 2 * p.C - 1);
  if (c0 >= c1) return;  // whole in one block, which wrote it
  const int r = (i - rg * tokens) * p.G + hq % p.G;
  // the first block may have begun before this segment; the others begin inside it
  auto part = [&](int c) { return (size_t)(c == c0 ? first : 2 * c) * p.RT + r; };
  float M = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.ml_part[part(c)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float sum = 0.f, a[E];
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll 4
  for (int c = c0 + (WIDE ? warp : 0); c <= c1; c += STEP) {
    const size_t at = part(c);
    const float2 y = p.ml_part[at];
    const float w = y.x == -INFINITY ? 0.f : ex2(y.x - M);
    sum = fmaf(w, y.y, sum);
    const float* o = p.o_part + at * D + E * lane;
    float v[E];
    if constexpr (E == 4) {
      const float4 t = *reinterpret_cast<const float4*>(o);
      v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
      const float2 t = *reinterpret_cast<const float2*>(o);
      v[0] = t.x, v[1] = t.y;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = fmaf(w, v[e], a[e]);
  }
  if (WIDE) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[warp][E * lane + e] = a[e];
    if (lane == 0) tot[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll
    for (int w = 0; w < MW; ++w) {
      sum += tot[w];
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] += acc[w][E * lane + e];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(p.out + (size_t)row * D + E * lane);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = __floats2bfloat162_rn(a[e] * inv, a[e + 1] * inv);
  if (lane == 0) p.lse[((size_t)b * p.Hq + hq) * p.T + i] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * LN2;
}

// How a shape is cut: rows of a few-rows block (0: the many-rows kernel), row
// tiles per block, tokens per row tile, row groups, rows per group and blocks.
struct Plan {
  int few, nq, tok, RG, RT, C;
};
static long long units_of(const Plan& x, int B, int Hkv, int cap) {
  return (long long)B * Hkv * x.RG * (((long long)cap + BK - 1) / BK);
}
static Plan plan(int B, int T, int Hq, int Hkv, int cap, int sms) {
  Plan x{};
  const int G = Hq / Hkv, R = G * T;
  x.few = R <= 16 ? 16 : R <= 32 ? 32 : 0;
  x.nq = R <= BM ? 1 : 2;
  x.tok = R <= BM ? T : BM / G;
  x.RG = (T + x.nq * x.tok - 1) / (x.nq * x.tok);
  x.RT = G * x.nq * x.tok;
  const long long units = units_of(x, B, Hkv, cap);
  x.C = (int)(units < sms ? units : sms);
  return x;
}
static bool supported(int B, int T, int Hq, int Hkv, int cap, int d) {
  return (d == 64 || d == 128) && T <= TMAX && Hq / Hkv <= BM && B <= ssa::MAX_SEQS &&
         (long long)B * Hkv <= (1 << 24) && cap <= (1 << 30) && (long long)B * T * Hq <= 0x7fffffff;
}
static bool positive(int B, int T, int Hq, int Hkv, int cap, int d) {
  return B > 0 && T > 0 && Hq > 0 && Hkv > 0 && cap > 0 && d > 0 && Hq % Hkv == 0;
}
static size_t table_bytes(const Plan& x, int B, int Hkv) { return (size_t)B * Hkv * x.RG * sizeof(int4); }
static size_t scratch_bytes(const Plan& x, int B, int Hkv, int d) {
  return table_bytes(x, B, Hkv) + (size_t)2 * x.C * x.RT * (d + 2) * sizeof(float);
}

static int device_sms(int* dev, int* sms) {
  return cudaGetDevice(dev) == cudaSuccess &&
                 cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) == cudaSuccess && *sms > 0
             ? SSA_OK
             : SSA_ERR_CUDA;
}

template <class Kernel>
static int launch(Kernel* kernel, size_t smem, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                  const Params& p, cudaStream_t st) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SSA_ERR_CUDA;
  kernel<<<p.C, NT, smem, st>>>(q, k, v, p);
  return cudaGetLastError() == cudaSuccess ? SSA_OK : SSA_ERR_CUDA;
}

template <int D>
static int run(const Plan& x, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const Params& p,
               cudaStream_t st) {
  int rc;
  switch (x.few) {
    case 16: rc = launch(tree_few_kernel<D, 16>, FewSmem<D, 16>::TOTAL, q, k, v, p, st); break;
    case 32: rc = launch(tree_few_kernel<D, 32>, FewSmem<D, 32>::TOTAL, q, k, v, p, st); break;
    default:
      rc = x.nq == 1 ? launch(tree_many_kernel<D, 1>, ManySmem<D, 1>::TOTAL, q, k, v, p, st)
                     : launch(tree_many_kernel<D, 2>, ManySmem<D, 2>::TOTAL, q, k, v, p, st);
  }
  if (rc != SSA_OK) return rc;
  // the merge's blocks may start once every block of the first kernel has; they wait for its results
  const long long rows = (long long)p.B * p.T * p.Hq;
  // a block a row: more than eight parts a row, and so few rows that a warp each would leave the GPU empty
  const bool wide = p.C > 8 * (long long)p.B * p.Hkv * p.RG && rows <= 8 * (long long)p.C;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + MW - 1) / MW));
  cfg.blockDim = dim3(32 * MW);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int tokens = x.nq * p.tok;
  const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, true>, p, tokens)
                             : cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, false>, p, tokens);
  return e == cudaSuccess ? SSA_OK : SSA_ERR_CUDA;
}

}  // namespace ssa_tree

extern "C" {

size_t ssa_decode_tree_workspace_bytes(int B, int T, int Hq, int Hkv, int cap, int d) {
  using namespace ssa_tree;
  int dev = 0, sms = 0;
  if (!positive(B, T, Hq, Hkv, cap, d) || !supported(B, T, Hq, Hkv, cap, d) || device_sms(&dev, &sms) != SSA_OK)
    return 0;
  return scratch_bytes(plan(B, T, Hq, Hkv, cap, sms), B, Hkv, d);
}

int ssa_decode_tree(const void* q, const void* k, const void* v, void* out, float* lse, const int32_t* lens,
                    const uint32_t* tree_mask, int B, int T, int Hq, int Hkv, int cap, int d, float scale,
                    void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ssa_tree;
  if (!q || !k || !v || !out || !lse || !lens || !tree_mask || !workspace) return SSA_ERR_INVALID_ARG;
  if (!positive(B, T, Hq, Hkv, cap, d)) return SSA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace)) & 15u)
    return SSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(lens) |
       reinterpret_cast<uintptr_t>(tree_mask)) & 3u)
    return SSA_ERR_INVALID_ARG;
  if (!supported(B, T, Hq, Hkv, cap, d)) return SSA_ERR_UNSUPPORTED;
  const size_t rows = (size_t)B * T * Hq, cache = (size_t)B * cap * Hkv * d * 2;
  const ssa::Span span[8] = {{out, rows * d * 2}, {lse, rows * 4}, {workspace, workspace_bytes}, {q, rows * d * 2},
                             {k, cache}, {v, cache}, {lens, (size_t)B * 4}, {tree_mask, (size_t)B * T * ((T + 31) / 32) * 4}};
  for (int i = 0; i < 3; ++i)  // each output against every other tensor
    for (int j = i + 1; j < 8; ++j)
      if (ssa::overlap(span[i], span[j])) return SSA_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != SSA_OK) return SSA_ERR_CUDA;
  const Plan x = plan(B, T, Hq, Hkv, cap, sms);
  if (units_of(x, B, Hkv, cap) > 0x7fffffff) return SSA_ERR_UNSUPPORTED;
  if (workspace_bytes < scratch_bytes(x, B, Hkv, d)) return SSA_ERR_INVALID_ARG;
  Params p{};
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.lens = lens;
  p.mask = tree_mask;
  p.segs = static_cast<int4*>(workspace);
  p.o_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + table_bytes(x, B, Hkv));
  p.ml_part = reinterpret_cast<float2*>(p.o_part + (size_t)2 * x.C * x.RT * d);
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.cap = cap;
  p.words = (T + 31) / 32;
  p.tok = x.tok;
  p.RG = x.RG;
  p.RT = x.RT;
  p.C = x.C;
  p.c = (float)((double)scale * 1.4426950408889634);
  p.stream_kv = x.RG == 1;
  p.status = ssa::device_status_word(dev);
  if (!p.status) return SSA_ERR_CUDA;
  p.wait_ns = ssa::wait_timeout_ns();
  CUtensorMap mq, mk, mv;
  if (!ssa::tma_map_bf16_box(&mq, q, B, T, Hq, d, p.G, x.tok) ||
      !ssa::tma_map_bf16(&mk, k, B, cap, Hkv, d, BK) || !ssa::tma_map_bf16(&mv, v, B, cap, Hkv, d, BK))
    return SSA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? run<128>(x, mq, mk, mv, p, st) : run<64>(x, mq, mk, mv, p, st);
}

}  // extern "C"
