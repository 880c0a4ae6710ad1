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
// Query rows are packed token-major, row (i - first) * G + g, into 128-row
// tiles.  Warps: 0 loads K and V; 1 issues S = Q K^T and O += P V (tcgen05, P as
// bf16 in TMEM over its S); 2 loads Q; 3 makes V safe; 4-7 and 8-11 are two
// softmax groups, a thread a row, each with its own S, P and O in TMEM.
//   NQ = 1 (one row tile): the groups take alternate key tiles of the same
//     rows, so one's products run under the other's exponentials; their
//     accumulators are added at the end of a segment, both of them reading the
//     half of the columns that they write.
//   NQ = 2 (two row tiles): each group has its own row tile, every key tile
//     is loaded once for both.
// More than two row tiles repeat the walk over the keys.
//
// Values that a row must not see: a hidden score becomes -inf, so P = 0; but
// 0 * inf and 0 * NaN are NaN, so warp 3 writes zeros over V rows past the last
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
constexpr int BM = 128;  // rows per row tile
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
  int* status;
  unsigned long long wait_ns;
  int B, T, Hq, Hkv, G, cap, words;
  int tok, RG, RT, nw;  // tokens per row tile, row groups, rows per group, warps with rows per softmax group
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

template <int D, int NQ>
struct Smem {
  static constexpr uint32_t Q_BYTES = BM * D * 2;  // a row tile
  static constexpr uint32_t KV_BYTES = BK * D * 2;
  static constexpr int FIT = (int)((200 * 1024 - NQ * Q_BYTES) / KV_BYTES);  // K and V tiles
  static constexpr int KST = (FIT + 1) / 2 < 4 ? (FIT + 1) / 2 : 4;
  static constexpr int VST = FIT / 2 < 4 ? FIT / 2 : 4;
  static constexpr uint32_t TOTAL = 1024 + NQ * Q_BYTES + (KST + VST) * KV_BYTES;
};

template <int D, int NQ>
__global__ void __launch_bounds__(NT, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using L = Smem<D, NQ>;
  constexpr int KST = L::KST, VST = L::VST;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t kfull[KST], kempty[KST], vfull[VST], vempty[VST], vsafe[VST];
  __shared__ uint64_t q_full, q_empty, s_full[2], p_ready[2], o_done, o_empty, ml_full[2], done;
  __shared__ float2 ml[2][2][BM];
  __shared__ uint32_t bad[NBAD][TMAX / 32];
  __shared__ int pref[ssa::MAX_SEQS + 1];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_s = smem_u32(base), k_s = q_s + NQ * L::Q_BYTES, v_s = k_s + KST * L::KV_BYTES;

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
    mbar_init(smem_u32(&o_empty), 2 * p.nw);
    mbar_init(smem_u32(&done), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_ready[i]), p.nw);
      mbar_init(smem_u32(&ml_full[i]), 2 * p.nw);
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
    if (lane == 0) {
      ssa::tma_prefetch_desc(&tm_k);
      ssa::tma_prefetch_desc(&tm_v);
      const uint64_t policy = ssa::l2_evict_first_policy();
      auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int hkv, int j0, int b) {
        mbar_arrive_expect_tx(bar, L::KV_BYTES);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          if (p.stream_kv) ssa::tma_load_4d_hint(dst + c * BK * 128, map, bar, c * 64, hkv, j0, b, policy);
          else ssa::tma_load_4d(dst + c * BK * 128, map, bar, c * 64, hkv, j0, b);
        }
      };
      int g = 0, kdone = 0, vdone = 0;
      bool ok = true;
      while (ok && walk.next(s))
        for (int t = 0; t < s.nt; ++t, ++g) {
          const int ks = g % KST, vs = g % VST, hkv = s.in / p.RG, j0 = (s.kt0 + t) * BK;
          ok = wait(&kempty[ks], ((g / KST) & 1) ^ 1);
          if (!ok) break;
          load(k_s + ks * L::KV_BYTES, &tm_k, smem_u32(&kfull[ks]), hkv, j0, s.b);
          kdone = g + 1;
          ok = wait(&vempty[vs], ((g / VST) & 1) ^ 1);
          if (!ok) break;
          load(v_s + vs * L::KV_BYTES, &tm_v, smem_u32(&vfull[vs]), hkv, j0, s.b);
          vdone = g + 1;
        }
      // nothing in flight when the block ends
      for (int t = max(0, kdone - KST); t < kdone; ++t)
        ssa::mbar_wait(smem_u32(&kfull[t % KST]), (t / KST) & 1, DRAIN_NS);
      for (int t = max(0, vdone - VST); t < vdone; ++t)
        ssa::mbar_wait(smem_u32(&vfull[t % VST]), (t / VST) & 1, DRAIN_NS);
    }
  } else if (warp == 1) {
    if (lane == 0) {
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
        if (t_s == 0 && !wait(&q_full, n_s & 1)) return false;
        if (!wait(&kfull[ks], (g / KST) & 1)) return false;
        ssa::tc_fence_after();
#pragma unroll
        for (int k16 = 0; k16 < D / 16; ++k16) {
          const uint32_t o = (k16 >> 2) * (128 * 128) + (k16 & 3) * 32;
          ssa::mma_ss(tmem + 256 * w, ssa::smem_desc_sw128(q_s + (NQ == 2 ? w : 0) * L::Q_BYTES + o, 16, 1024),
                      ssa::smem_desc_sw128(k_s + ks * L::KV_BYTES + o, 16, 1024), idesc_qk, k16 > 0);
        }
        ssa::mma_commit(smem_u32(&s_full[w]));
        if ((h_s + 1) % NQ == 0) ssa::mma_commit(smem_u32(&kempty[ks]));
        ++h_s;
        if (++t_s == ss.nt * NQ) {
          ssa::mma_commit(smem_u32(&q_empty));
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
          if (!wait(&p_ready[w], (h >> 1) & 1) || !wait(&vfull[vs], (g / VST) & 1) ||
              !wait(&vsafe[vs], (g / VST) & 1) || (t == 0 && !wait(&o_empty, (n & 1) ^ 1))) {
            ok = false;
            break;
          }
          ssa::tc_fence_after();
#pragma unroll
          for (int k16 = 0; k16 < BK / 16; ++k16) {
            ssa::mma_ts(tmem + 256 * w + 128, tmem + 256 * w + k16 * 8,
                        ssa::smem_desc_sw128(v_s + vs * L::KV_BYTES + k16 * 16 * 128, BK * 128, 1024), idesc_pv, acc[w]);
            acc[w] = 1u;
          }
          if ((h + 1) % NQ == 0) ssa::mma_commit(smem_u32(&vempty[vs]));
          if (t == s.nt * NQ - 1) ssa::mma_commit(smem_u32(&o_done));
          if (more) ok = issue_s();
        }
        ++n;
      }
      ssa::mma_commit(smem_u32(&done));
      ssa::mbar_wait(smem_u32(&done), 0, DRAIN_NS);  // no MMA in flight when TMEM is freed
    }
  } else if (warp == 2) {
    if (lane == 0) {
      const int tokens = NQ == 1 ? p.T : p.tok;
      int n = 0;
      while (walk.next(s)) {
        if (!wait(&q_empty, (n & 1) ^ 1)) break;
        mbar_arrive_expect_tx(smem_u32(&q_full), (uint32_t)(NQ * p.G * tokens * D * 2));
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
    // V rows that not every row sees.  (Element positions are swizzled within
    // a row's 128-byte pieces; what is done here does not depend on them.)
    int g = 0, n = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const int len = clamp_len(p.lens, s.b, p.cap), keys = key_count(p, s.b);
      if (lane < TMAX / 32) bad[n % NBAD][lane] = 0u;
      __syncwarp();
      for (int t = 0; t < s.nt; ++t, ++g) {
        const int vs = g % VST, j0 = (s.kt0 + t) * BK;
        ok = __all_sync(0xffffffffu, wait(&vfull[vs], (g / VST) & 1));
        if (!ok) break;
        if (j0 + BK > len) {
          uint8_t* tile = base + NQ * L::Q_BYTES + KST * L::KV_BYTES + vs * L::KV_BYTES;
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
  } else if ((warp & 3) < p.nw) {
    const int wg = (warp - 4) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = lanes + 256 * wg, o_col = s_col + 128;
    const int row = (warp & 3) * 32 + lane;
    const float c = p.c;
    const uint64_t c2 = ssa::f2_pack(c, c);
    int g = 0, n = 0;
    uint32_t cnt = 0;  // S tiles of this group so far
    bool ok = true;
    while (ok && walk.next(s)) {
      const int len = clamp_len(p.lens, s.b, p.cap), tb = min(p.T, p.cap - len);
      const int hkv = s.in / p.RG, rg = s.in % p.RG;
      const int i = rg * (NQ * p.tok) + (NQ == 2 ? wg * p.tok : 0) + row / p.G, hq = hkv * p.G + row % p.G;
      const bool valid = row < p.G * p.tok && i < p.T;
      const uint32_t* mrow = p.mask + ((size_t)s.b * p.T + (valid ? i : 0)) * p.words;
      float m = -INFINITY, l = 0.f;  // max in use (of q.k), sum
      bool any = false;
      for (int t = 0; t < s.nt; ++t) {
        if (NQ == 1 && ((g + t) & 1) != wg) continue;
        ok = __all_sync(0xffffffffu, wait(&s_full[wg], cnt & 1));
        if (!ok) break;
        ++cnt;
        ssa::tc_fence_after();
        float x[BK];
        ssa::tmem_ld64f(s_col, x);
        ssa::tmem_ld64f(s_col + 64, x + 64);
        ssa::tmem_wait_ld();
        const int j0 = (s.kt0 + t) * BK;
        if (j0 + BK > len) {
#pragma unroll
          for (int w = 0; w < BK / 32; ++w) {
            const uint32_t see = valid ? sees32(mrow, j0 + 32 * w - len, tb) : 0u;
#pragma unroll
            for (int e = 0; e < 32; ++e) x[32 * w + e] = (see >> e) & 1u ? x[32 * w + e] : -INFINITY;
          }
        }
        float a0 = fmaxf(x[0], x[1]), a1 = fmaxf(x[2], x[3]);
#pragma unroll
        for (int e = 4; e < BK; e += 4) {
          a0 = ssa::fmax3(a0, x[e], x[e + 1]);
          a1 = ssa::fmax3(a1, x[e + 2], x[e + 3]);
        }
        const float tmax = fmaxf(a0, a1);
        // The max in use only follows when it is more than 2^8 behind: P stays
        // below 2^8 and the sums in fp32, and O is rarely rescaled.
        if (!any) {
          m = tmax;
          any = true;
        } else if (__any_sync(0xffffffffu, tmax * c > m * c + 8.f)) {
          // (S of this tile is complete, so the P V before it is too)
          const bool up = tmax > m;
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
        for (int h = 0; h < BK / 32; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float p0, p1;
            ssa::f2_unpack(ssa::ffma2(ssa::f2_pack(x[32 * h + 2 * e], x[32 * h + 2 * e + 1]), c2, mc2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum[e & 1] = ssa::fadd2(sum[e & 1], ssa::f2_pack(p0, p1));
            // rounded to bf16 for the tensor cores; the sum takes the unrounded ones
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
            pk[e] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          ssa::tmem_st16(s_col + 16 * h, pk);
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
      g += s.nt;
      if (!ok) break;

      // ---- end of the segment
      float w0 = 1.f, w1 = 0.f;  // weights of this group's accumulator and of the other's
      bool other = false;
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
        // the same sum in both groups, to the bit
        l = wg == 0 ? fmaf(l, w0, y.y * w1) : fmaf(y.y, w1, l * w0);
        other = s.nt > 1 || !any;
      }
      ok = __all_sync(0xffffffffu, wait(&o_done, n & 1));
      if (!ok) break;
      ssa::tc_fence_after();
      const bool whole = s.nt == s.tiles;
      const int slot = 2 * blockIdx.x + (n > 0 ? 1 : 0);  // a part is a block's first or its last segment
      const size_t part = (size_t)slot * p.RT + (NQ == 2 ? wg * p.tok * p.G : 0) + row;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      constexpr int COLS = NQ == 1 ? D / 2 : D;
      const int col0 = NQ == 1 ? wg * (D / 2) : 0;
      const uint32_t o_other = lanes + 256 * (wg ^ 1) + 128;
      const uint32_t* bd = bad[n % NBAD];
      const bool fix = (bd[0] | bd[1] | bd[2] | bd[3]) != 0u;
#pragma unroll 1
      for (int cc = 0; cc < COLS / 32; ++cc) {
        float o[32];
        if (any) {
          ssa::tmem_ld32f(o_col + col0 + 32 * cc, o);
          ssa::tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = any ? o[e] * w0 : 0.f;
        if (other) {
          float y[32];
          ssa::tmem_ld32f(o_other + col0 + 32 * cc, y);
          ssa::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(y[e], w1, o[e]);
        }
        if (cc == COLS / 32 - 1) {  // O is in registers: the next segment may overwrite it
          ssa::tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&o_empty));
        }
        if (!valid) continue;
        if (fix) {
#pragma unroll 1
          for (int t = 0; t < tb; ++t) {
            if (!((bd[t >> 5] >> (t & 31)) & 1u) || !((mask_word(mrow, t >> 5, tb) >> (t & 31)) & 1u)) continue;
            const __nv_bfloat16* v =
                p.v + (((size_t)s.b * p.cap + len + t) * p.Hkv + hkv) * D + col0 + 32 * cc;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float y = __bfloat162float(v[e]);
              if (!isfinite(y)) o[e] += y;
            }
          }
        }
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + (((size_t)s.b * p.T + i) * p.Hq + hq) * D + col0 + 32 * cc);
#pragma unroll
          for (int e8 = 0; e8 < 4; ++e8) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b2 =
                  __floats2bfloat162_rn(o[8 * e8 + 2 * e] * inv, o[8 * e8 + 2 * e + 1] * inv);
              u[e] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            dst[e8] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(p.o_part + part * D + col0 + 32 * cc);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (valid && (NQ == 2 || wg == 0)) {
        if (whole) p.lse[((size_t)s.b * p.Hq + hq) * p.T + i] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * LN2;
        else p.ml_part[part] = make_float2(m * c, l);
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

// One block a query row: the parts of its (sequence, key head, row group) in
// block order, every CW-th by a warp, D / 32 columns a lane.
constexpr int CW = 8;

template <int D>
__global__ void __launch_bounds__(32 * CW) tree_merge_kernel(const __grid_constant__ Params p, int tokens) {
  constexpr int E = D / 32;
  __shared__ float acc[CW][D];
  __shared__ float2 top[CW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = blockIdx.x % p.Hq, bi = blockIdx.x / p.Hq, i = bi % p.T, b = bi / p.T;
  const int rg = i / tokens, in = hq / p.G * p.RG + rg, inner = p.Hkv * p.RG;
  const int tiles = tile_count(p, b);
  long long before = 0, all = 0;
  for (int x = lane; x < p.B; x += 32) {
    const int n = tile_count(p, x);
    all += n;
    if (x < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  const long long U = all * inner, u0 = before * inner + (long long)in * tiles;
  const int C = (int)(p.C < U ? p.C : U);
  // block of unit u: the largest c with U c / C <= u
  const int c0 = (int)(((u0 + 1) * C - 1) / U), c1 = (int)(((u0 + tiles) * C - 1) / U);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // by every block: what follows in the stream needs both kernels
  if (c0 == c1) return;  // whole in one block, which wrote it
  const int r = (i - rg * tokens) * p.G + hq % p.G;
  // block c0 may have begun before this segment; the others begin inside it
  const size_t first = 2 * (size_t)c0 + (ssa::range_start(U, c0, C) < u0 ? 1 : 0);
  auto part = [&](int c) { return (c == c0 ? first : 2 * (size_t)c) * p.RT + r; };
  float M = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.ml_part[part(c)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float sum = 0.f, a[E];
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += CW) {
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
#pragma unroll
  for (int e = 0; e < E; ++e) acc[warp][E * lane + e] = a[e];
  if (lane == 0) top[warp] = make_float2(M, sum);
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  float x0 = 0.f, x1 = 0.f;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < CW; ++w) {
    sum += top[w].y;
    x0 += acc[w][2 * threadIdx.x];
    x1 += acc[w][2 * threadIdx.x + 1];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<__nv_bfloat162*>(p.out + (size_t)blockIdx.x * D + 2 * threadIdx.x) =
      __floats2bfloat162_rn(x0 * inv, x1 * inv);
  if (threadIdx.x == 0)
    p.lse[((size_t)b * p.Hq + hq) * p.T + i] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * LN2;
}

// How a shape is cut: tokens per row tile, row tiles per block, row groups, rows
// per group and blocks.
struct Plan {
  int tok, nq, RG, RT, C;
};
static Plan plan(int B, int T, int Hq, int Hkv, int cap, int sms) {
  Plan x{};
  const int G = Hq / Hkv;
  x.tok = BM / G;
  x.nq = T <= x.tok ? 1 : 2;
  x.RG = (T + x.nq * x.tok - 1) / (x.nq * x.tok);
  x.RT = G * (x.nq == 1 ? T : 2 * x.tok);
  const long long units = (long long)B * Hkv * x.RG * (((long long)cap + BK - 1) / BK);
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
static size_t part_bytes(const Plan& x, int d) { return (size_t)2 * x.C * x.RT * (d + 2) * sizeof(float); }

static int device_sms(int* dev, int* sms) {
  return cudaGetDevice(dev) == cudaSuccess &&
                 cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) == cudaSuccess && *sms > 0
             ? SSA_OK
             : SSA_ERR_CUDA;
}

template <int D, int NQ>
static int launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const Params& p, cudaStream_t st) {
  if (cudaFuncSetAttribute(tree_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)Smem<D, NQ>::TOTAL) != cudaSuccess)
    return SSA_ERR_CUDA;
  tree_kernel<D, NQ><<<p.C, NT, Smem<D, NQ>::TOTAL, st>>>(q, k, v, p);
  if (cudaGetLastError() != cudaSuccess) return SSA_ERR_CUDA;
  // its blocks may start once every block of the first kernel has; they wait for its results
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.B * p.T * p.Hq));
  cfg.blockDim = dim3(32 * CW);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, p, NQ * p.tok) == cudaSuccess ? SSA_OK : SSA_ERR_CUDA;
}

}  // namespace ssa_tree

extern "C" {

size_t ssa_decode_tree_workspace_bytes(int B, int T, int Hq, int Hkv, int cap, int d) {
  using namespace ssa_tree;
  int dev = 0, sms = 0;
  if (!positive(B, T, Hq, Hkv, cap, d) || !supported(B, T, Hq, Hkv, cap, d) || device_sms(&dev, &sms) != SSA_OK)
    return 0;
  return part_bytes(plan(B, T, Hq, Hkv, cap, sms), d);
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
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != SSA_OK) return SSA_ERR_CUDA;
  const Plan x = plan(B, T, Hq, Hkv, cap, sms);
  if (workspace_bytes < part_bytes(x, d)) return SSA_ERR_INVALID_ARG;
  Params p{};
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.lens = lens;
  p.mask = tree_mask;
  p.o_part = static_cast<float*>(workspace);
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
  p.nw = ((x.nq == 1 ? x.RT : x.RT / 2) + 31) / 32;
  p.C = x.C;
  p.c = (float)((double)scale * 1.4426950408889634);
  p.stream_kv = x.RG == 1;
  p.status = ssa::device_status_word(dev);
  if (!p.status) return SSA_ERR_CUDA;
  p.wait_ns = ssa::wait_timeout_ns();
  CUtensorMap mq, mk, mv;
  if (!ssa::tma_map_bf16_box(&mq, q, B, T, Hq, d, p.G, x.nq == 1 ? T : x.tok) ||
      !ssa::tma_map_bf16(&mk, k, B, cap, Hkv, d, BK) || !ssa::tma_map_bf16(&mv, v, B, cap, Hkv, d, BK))
    return SSA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d == 128) return x.nq == 1 ? launch<128, 1>(mq, mk, mv, p, st) : launch<128, 2>(mq, mk, mv, p, st);
  return x.nq == 1 ? launch<64, 1>(mq, mk, mv, p, st) : launch<64, 2>(mq, mk, mv, p, st);
}

}  // extern "C"
