// ssa_cache.cu -- writing and compacting a key/value cache on B200 (sm_100a):
// ssa_cache_append (per-head norm, position rotation, append) and
// ssa_cache_evict (selection of the heaviest keys, compaction).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/ssa_cache.h"
#include "internal.h"

namespace ssa_cache {

namespace cg = cooperative_groups;

// ============================================================ append

// Streaming work: every q, k, v value is read once and written once, bound by
// HBM.  One warp takes one token and a range of its heads, D / 8 lanes a head
// row (16 bytes a lane), so the angles of the token (two to eight sine/cosine
// pairs a lane) are computed once in registers and serve all of its heads; the
// norm is a shuffle reduction inside the row's lanes and the rotation partner,
// half a rotated width away, comes by shuffle.  The next AU head rows are on their
// way while the current ones are computed: 75,600 tokens of 40 + 40 + 40 heads take
// 717 us (6.5 TB/s, the rate of a copy; 1,055 without the look-ahead).  A smaller
// register budget (spills), warps that go on to further tokens and angles shared
// through shared memory all measured the same or slower.
constexpr int AW = 4;  // warps per block
constexpr int AU = 4;  // head rows a lane group loads at once

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t st[9];  // batch, token, head strides of q, k, v (elements)
  const float *wq, *wk;
  const int32_t *pos, *start, *count;
  __nv_bfloat16 *q_out, *k_cache, *v_cache;
  float eps, factor;
  int axes, rot, L, Hq, Hkv, cap;
  int chunks, per;  // warps per token, heads per warp
  int64_t n_warps;
  uint64_t freq[64];  // turns per position, modulo 1, in units of 2^-64
  uint8_t axis[64];
};

template <int D, bool PAIRS>
__global__ void __launch_bounds__(32 * AW) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LH = D / 8, RP = 32 / LH;  // lanes per head row, rows per warp
  const int lane = threadIdx.x & 31, u = lane % LH, sub = lane / LH;
  const int64_t gw = (int64_t)blockIdx.x * AW + (threadIdx.x >> 5);
  if (gw >= p.n_warps) return;
  const int64_t tok = gw / p.chunks;
  const int chunk = (int)(gw % p.chunks);
  const int64_t b = tok / p.L;
  const int i = (int)(tok % p.L);
  if (p.count != nullptr && i >= p.count[b]) return;
  const int64_t row = (p.start != nullptr ? p.start[b] : 0) + (int64_t)i;
  const bool in_cache = row >= 0 && row < p.cap;

  // cosine and signed sine of this lane's columns [8u, 8u + 8).  The angle in
  // turns is pos * freq modulo 1: a 64-bit integer product, exact, so only the
  // top 32 bits' conversion to fp32 rounds, whatever the position.
  const bool turns = 8 * u < p.rot;
  const int half = p.rot / 2;
  constexpr int NA = PAIRS ? 4 : 8;
  float cs[NA], sn[NA];
#pragma unroll
  for (int e = 0; e < NA; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }
  if (turns) {
    const int p0 = PAIRS ? 4 * u : (8 * u < half ? 8 * u : 8 * u - half);
    const float sign = (!PAIRS && 8 * u < half) ? -1.f : 1.f;
    const int32_t* pos = p.pos + tok * p.axes;
#pragma unroll
    for (int e = 0; e < NA; ++e) {
      const uint64_t t = (uint64_t)(int64_t)pos[p.axis[p0 + e]] * p.freq[p0 + e];
      float s, c;
      sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
      cs[e] = c * p.factor;
      sn[e] = s * p.factor * sign;
    }
  }
  const int from = PAIRS || !turns ? lane : (8 * u < half ? lane + half / 8 : lane - half / 8);

  // Head rows [h0, h1) of one tensor: src and dst at this lane's columns of head 0.
  auto rows = [&](int h0, int h1, const __nv_bfloat16* src, int64_t step, __nv_bfloat16* dst, const float* w, bool plain) {
    if (h0 >= h1) return;
    float wt[8];
    if (w != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) wt[e] = w[8 * u + e];  // (4-byte aligned)
    }
    uint4 next[AU];
    auto load = [&](int h) {
#pragma unroll
      for (int a = 0; a < AU; ++a) {
        const int at = h + a * RP + sub;
        next[a] = make_uint4(0u, 0u, 0u, 0u);
        if (at < h1) next[a] = __ldcs(reinterpret_cast<const uint4*>(src + at * step));
      }
    };
    load(h0);
#pragma unroll 1
    for (int h = h0; h < h1; h += RP * AU) {
      uint4 raw[AU];
#pragma unroll
      for (int a = 0; a < AU; ++a) raw[a] = next[a];
      if (h + RP * AU < h1) load(h + RP * AU);
#pragma unroll
      for (int a = 0; a < AU; ++a) {
        if (h + a * RP >= h1) break;  // warp-uniform
        const int at = h + a * RP + sub;
        if (!plain) {
          float x[8];
          uint32_t* r = &raw[a].x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(r[e] << 16);
            x[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
          }
          if (w != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float g = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= g * wt[e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y0, y1;
            if (PAIRS) {
              y0 = x[2 * e] * cs[e] - x[2 * e + 1] * sn[e];
              y1 = x[2 * e + 1] * cs[e] + x[2 * e] * sn[e];
            } else {
              y0 = fmaf(x[2 * e], cs[2 * e % NA], __shfl_sync(0xffffffffu, x[2 * e], from) * sn[2 * e % NA]);
              y1 = fmaf(x[2 * e + 1], cs[(2 * e + 1) % NA],
                        __shfl_sync(0xffffffffu, x[2 * e + 1], from) * sn[(2 * e + 1) % NA]);
            }
            const __nv_bfloat162 t = turns ? __floats2bfloat162_rn(y0, y1) : __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            r[e] = *reinterpret_cast<const uint32_t*>(&t);
          }
        }
        if (at < h1) *reinterpret_cast<uint4*>(dst + at * D) = raw[a];
      }
    }
  };
  const int lo = chunk * p.per, hi = min(p.Hq + 2 * p.Hkv, lo + p.per);
  const int64_t cell = (b * p.cap + row) * p.Hkv * D + 8 * u;
  rows(lo, min(hi, p.Hq), p.q + b * p.st[0] + i * p.st[1] + 8 * u, p.st[2], p.q_out + tok * p.Hq * D + 8 * u, p.wq, false);
  if (!in_cache) return;
  rows(max(lo - p.Hq, 0), min(hi - p.Hq, p.Hkv), p.k + b * p.st[3] + i * p.st[4] + 8 * u, p.st[5], p.k_cache + cell, p.wk,
       false);
  rows(max(lo - p.Hq - p.Hkv, 0), min(hi - p.Hq - p.Hkv, p.Hkv), p.v + b * p.st[6] + i * p.st[7] + 8 * u, p.st[8],
       p.v_cache + cell, nullptr, true);
}

// ============================================================ evict

// Selection: the m-th largest mass of a (sequence, key head) by radix select
// over order-preserving 32-bit keys (digits of 11, 11 and 10 bits), then an
// ordered compaction, in one launch.  A cluster of up to 8 blocks shares one
// (sequence, key head), each holding its slice of the keys in shared memory, so
// the masses are read once; the blocks' histograms are added through distributed
// shared memory.  Counts are integers and positions come from prefix sums in
// index order, so ties go to the lower index whatever the blocks' order.  64 lists of
// 31k masses, 4,096 of each chosen: 24 us (10 us at 700 masses: the passes' own
// latency); four copies of the first histogram, against collisions, changed nothing.
constexpr int ST = 1024, SW = ST / 32;
constexpr int BINS = 2048;
constexpr int MU = 8, MP = 4;  // masses a thread loads at once: selection, compaction
constexpr int MAX_KEYS = 40960;  // keys of a block's slice kept in shared memory (160 KB)

struct EvictParams {
  const __nv_bfloat16 *k, *v;
  const float* mass;
  const int32_t* lens;
  __nv_bfloat16 *k_out, *v_out;
  float* mass_out;
  int32_t *index_out, *lens_out;
  int B, Hkv, cap, cap_out, keep, sink, recent;
  int max_keys;
};

// larger mass <-> larger key; -0 counts as 0 and NaN as the smallest
__device__ __forceinline__ uint32_t mass_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(ST, 1) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t s_keys[];
  __shared__ uint32_t s_hist[2][BINS];
  __shared__ uint32_t s_warp[SW], s_warp2[SW];
  __shared__ uint32_t s_digit, s_want;
  __shared__ uint32_t s_tot[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x / CS;
  const int b = seg / p.Hkv;
  const int n = min(max(p.lens[b], 0), p.cap);
  const float* mass = p.mass + (size_t)seg * p.cap;
  int32_t* index = p.index_out + (size_t)seg * p.keep;
  float* mass_out = p.mass_out + (size_t)seg * p.cap_out;
  const int kept = min(n, p.keep);
  if (seg % p.Hkv == 0 && rank == 0 && tid == 0) p.lens_out[b] = kept;
  const int t0 = rank * ST + tid, step = CS * ST;
  for (int j = kept + t0; j < p.cap_out; j += step) mass_out[j] = 0.f;
  if (n <= p.keep) {  // the same for every block of the cluster
    for (int j = t0; j < p.keep; j += step) index[j] = j < n ? j : -1;
    for (int j = t0; j < n; j += step) mass_out[j] = mass[j];
    return;
  }
  for (int j = t0; j < p.sink; j += step) {
    index[j] = j;
    mass_out[j] = mass[j];
  }
  for (int t = t0; t < p.recent; t += step) {
    const int at = p.keep - p.recent + t, j = n - p.recent + t;
    index[at] = j;
    mass_out[at] = mass[j];
  }
  const int m = p.keep - p.sink - p.recent;  // to choose among [sink, n - recent), which holds more than m
  if (m == 0) return;
  const int lo = p.sink, M = n - p.recent - p.sink;
  const int per = ((M + CS - 1) / CS + 31) & ~31;
  const int a = min(rank * per, M), len = min(per, M - a);  // this block's slice, relative to lo
  const float* mine = mass + lo + a;
  const bool cached = len <= p.max_keys;
  auto key = [&](int j) -> uint32_t { return cached ? s_keys[j] : mass_key(mine[j]); };

  uint32_t prefix = 0, want = (uint32_t)m;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t dmask = pass == 2 ? 1023u : 2047u;
    const uint32_t pmask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
    uint32_t* hist = s_hist[pass & 1];
    hist[tid] = 0u;
    hist[tid + ST] = 0u;
    __syncthreads();
    if (pass == 0 && cached) {
      for (int j0 = tid; j0 < len; j0 += MU * ST) {  // MU loads on their way at once
        float v[MU];
#pragma unroll
        for (int e = 0; e < MU; ++e) v[e] = j0 + e * ST < len ? mine[j0 + e * ST] : 0.f;
#pragma unroll
        for (int e = 0; e < MU; ++e) {
          if (j0 + e * ST >= len) break;
          const uint32_t x = mass_key(v[e]);
          s_keys[j0 + e * ST] = x;
          atomicAdd(&hist[x >> 21], 1u);
        }
      }
    } else {
      for (int j = tid; j < len; j += ST) {
        const uint32_t x = key(j);
        if ((x & pmask) == prefix) atomicAdd(&hist[(x >> shift) & dmask], 1u);
      }
    }
    // every block's histogram is complete.  (The buffers alternate: a block
    // clears one only after the barrier of the pass in between, which the
    // others reach once they have read it.)
    cluster.sync();
    // thread t: bins 2047 - 2t and 2046 - 2t, largest first
    uint32_t c0 = 0, c1 = 0;
    for (int r = 0; r < CS; ++r) {
      const uint32_t* h = cluster.map_shared_rank(hist, r);
      c0 += h[BINS - 1 - 2 * tid];
      c1 += h[BINS - 2 - 2 * tid];
    }
    uint32_t incl = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      uint32_t x = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += t;
      }
      s_warp[lane] = x;
    }
    __syncthreads();
    if (warp > 0) incl += s_warp[warp - 1];
    const uint32_t before = incl - c0 - c1;  // keys in larger bins
    if (before < want && want <= incl) {     // exactly one thread
      const bool second = want > before + c0;
      s_digit = (uint32_t)(BINS - 1 - 2 * tid) - (second ? 1u : 0u);
      s_want = want - before - (second ? c0 : 0u);
    }
    __syncthreads();
    prefix |= s_digit << shift;
    want = s_want;
    __syncthreads();
  }
  // taken: keys above `prefix`, and the first `want` of those equal to it.
  // Warp w owns a contiguous run of the slice.
  const int run = ((per / 32 + SW - 1) / SW) * 32;
  const int r0 = min(warp * run, len), r1 = min(r0 + run, len);
  uint32_t gt = 0, eq = 0;
  for (int j = r0; j < r1; j += 32) {
    const bool in = j + lane < r1;
    const uint32_t x = in ? key(j + lane) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, in && x > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, in && x == prefix));
  }
  if (lane == 0) {
    s_warp[warp] = gt;
    s_warp2[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t x = s_warp[lane], y = s_warp2[lane];
    const uint32_t x0 = x, y0 = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += t;
        y += v;
      }
    }
    s_warp[lane] = x - x0;
    s_warp2[lane] = y - y0;
    if (lane == 31) {
      s_tot[0] = x;
      s_tot[1] = y;
    }
  }
  cluster.sync();
  uint32_t g0 = s_warp[warp], e0 = s_warp2[warp];
  for (int r = 0; r < rank; ++r) {
    const uint32_t* t = cluster.map_shared_rank(s_tot, r);
    g0 += t[0];
    e0 += t[1];
  }
#pragma unroll 1
  for (int j4 = r0; j4 < r1; j4 += 32 * MP) {
    float v[MP];  // loaded for all of them, MP at once: a load for each taken one costs its latency every time
#pragma unroll
    for (int e = 0; e < MP; ++e) v[e] = j4 + 32 * e + lane < r1 ? mine[j4 + 32 * e + lane] : 0.f;
#pragma unroll
    for (int e = 0; e < MP; ++e) {
      const int j = j4 + 32 * e + lane;
      const bool in = j < r1;
      const uint32_t x = in ? (cached ? s_keys[j] : mass_key(v[e])) : 0u;
      const uint32_t bg = __ballot_sync(0xffffffffu, in && x > prefix);
      const uint32_t be = __ballot_sync(0xffffffffu, in && x == prefix);
      const uint32_t below = (1u << lane) - 1u;
      const uint32_t g = g0 + __popc(bg & below), q = e0 + __popc(be & below);
      if (in && (x > prefix || (x == prefix && q < want))) {
        const int at = p.sink + (int)(g + min(q, want));
        index[at] = lo + a + j;
        mass_out[at] = v[e];
      }
      g0 += __popc(bg);
      e0 += __popc(be);
    }
  }
  cluster.sync();  // the others may still read this block's totals
}

// Compaction: D / 8 lanes a row, key heads fastest (the output's order).  Launched
// early, it waits for the selection.
constexpr int GT = 256, GU = 2;

template <int D>
__global__ void __launch_bounds__(GT) evict_gather_kernel(const EvictParams p) {
  constexpr int LH = D / 8, ROWS = GT / LH;
  const int u = threadIdx.x % LH, g = threadIdx.x / LH;
  const int64_t total = (int64_t)p.B * p.keep * p.Hkv;
  uint4 kv[2 * GU];
  int64_t dst[GU];
  asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
  for (int a = 0; a < GU; ++a) {
    const int64_t r = ((int64_t)blockIdx.x * GU + a) * ROWS + g;
    dst[a] = -1;
    if (r < total) {
      const int h = (int)(r % p.Hkv);
      const int64_t s = r / p.Hkv;
      const int slot = (int)(s % p.keep);
      const int64_t b = s / p.keep;
      const int j = p.index_out[(b * p.Hkv + h) * p.keep + slot];
      if (j >= 0) {
        const int64_t at = ((b * p.cap + j) * p.Hkv + h) * D + 8 * u;
        kv[2 * a] = __ldcs(reinterpret_cast<const uint4*>(p.k + at));
        kv[2 * a + 1] = __ldcs(reinterpret_cast<const uint4*>(p.v + at));
        dst[a] = ((b * p.cap_out + slot) * p.Hkv + h) * D + 8 * u;
      }
    }
  }
#pragma unroll
  for (int a = 0; a < GU; ++a)
    if (dst[a] >= 0) {
      *reinterpret_cast<uint4*>(p.k_out + dst[a]) = kv[2 * a];
      *reinterpret_cast<uint4*>(p.v_out + dst[a]) = kv[2 * a + 1];
    }
}

static bool mis(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0; }

static int sm_count(int* out) {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
    return SSA_ERR_CUDA;
  *out = v;
  return SSA_OK;
}

}  // namespace ssa_cache

extern "C" {

int ssa_cache_append(const void* q, const void* k, const void* v, const int64_t* strides,
                     const float* q_weight, const float* k_weight, float eps, const int32_t* positions,
                     const double* inv_freq, const int32_t* axis, int axes, int rot, int interleaved,
                     float factor, const int32_t* start, const int32_t* count, void* q_out, void* k_cache,
                     void* v_cache, int B, int L, int Hq, int Hkv, int d, int cap, void* stream) {
  using namespace ssa_cache;
  if (!q || !k || !v || !strides || !q_out || !k_cache || !v_cache) return SSA_ERR_INVALID_ARG;
  if (B <= 0 || L <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || cap <= 0 || rot < 0) return SSA_ERR_INVALID_ARG;
  if (mis(q, 16) || mis(k, 16) || mis(v, 16) || mis(q_out, 16) || mis(k_cache, 16) || mis(v_cache, 16) ||
      mis(q_weight, 4) || mis(k_weight, 4) || mis(positions, 4) || mis(start, 4) || mis(count, 4))
    return SSA_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && (!(eps >= 0.f) || !std::isfinite(eps))) return SSA_ERR_INVALID_ARG;
  if (rot > 0 && (!positions || !inv_freq || !std::isfinite(factor))) return SSA_ERR_INVALID_ARG;
  for (int i = 0; i < 9; ++i)
    if (strides[i] < 0 || strides[i] % 8 != 0) return SSA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSA_ERR_UNSUPPORTED;
  if (rot % 16 != 0 || rot > d || axes < 1 || axes > 4) return SSA_ERR_UNSUPPORTED;
  const size_t cache_bytes = (size_t)B * cap * Hkv * d * 2, out_bytes = (size_t)B * L * Hq * d * 2;
  auto extent = [&](const int64_t* st, int heads) {
    return (size_t)((B - 1) * st[0] + (L - 1) * st[1] + (heads - 1) * st[2] + d) * 2;
  };
  const ssa::Span in[8] = {{q, extent(strides, Hq)},
                           {k, extent(strides + 3, Hkv)},
                           {v, extent(strides + 6, Hkv)},
                           {q_weight, (size_t)d * 4},
                           {k_weight, (size_t)d * 4},
                           {rot > 0 ? positions : nullptr, (size_t)B * L * axes * 4},
                           {start, (size_t)B * 4},
                           {count, (size_t)B * 4}};
  const ssa::Span made[3] = {{k_cache, cache_bytes}, {v_cache, cache_bytes}, {q_out, out_bytes}};
  const bool in_place = q_out == q && (Hq == 1 || strides[2] == d) && (L == 1 || strides[1] == (int64_t)Hq * d) &&
                        (B == 1 || strides[0] == (int64_t)L * Hq * d);
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 8; ++j)
      if (ssa::overlap(made[i], in[j]) && !(i == 2 && j == 0 && in_place)) return SSA_ERR_INVALID_ARG;
    if (ssa::overlap(made[i], made[(i + 1) % 3])) return SSA_ERR_INVALID_ARG;
  }
  AppendParams p{};
  for (int i = 0; i < rot / 2; ++i) {
    if (!std::isfinite(inv_freq[i])) return SSA_ERR_INVALID_ARG;
    if (axis && (axis[i] < 0 || axis[i] >= axes)) return SSA_ERR_INVALID_ARG;
    const long double turn = (long double)inv_freq[i] / 6.283185307179586476925286766559005768L;
    const long double frac = ldexpl(turn - floorl(turn), 64);
    p.freq[i] = frac < 18446744073709551615.0L ? (uint64_t)frac : 0u;  // 1 turn is 0
    p.axis[i] = (uint8_t)(axis ? axis[i] : 0);
  }
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  for (int i = 0; i < 9; ++i) p.st[i] = strides[i];
  p.wq = q_weight;
  p.wk = k_weight;
  p.pos = positions;
  p.start = start;
  p.count = count;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  p.eps = eps;
  p.factor = factor;
  p.axes = axes;
  p.rot = rot;
  p.L = L;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.cap = cap;
  int sms = 0;
  if (sm_count(&sms) != SSA_OK) return SSA_ERR_CUDA;
  // Few tokens: split a token's heads over warps until the GPU has about 16
  // warps an SM to hide latency with; many tokens: one warp a token, which computes
  // the angles once.  (64 or 128 warps an SM: 55 and 61 us against 49 at 8,192
  // tokens of 32 / 8 heads, since every warp computes them again.)
  const int rp = 32 / (d / 8), HT = Hq + 2 * Hkv;
  const int64_t tokens = (int64_t)B * L, most = (HT + rp - 1) / rp;
  int64_t chunks = ((int64_t)sms * 16 + tokens - 1) / tokens;
  if (chunks > most) chunks = most;
  const int64_t per = ((HT + chunks - 1) / chunks + rp - 1) / rp * rp;
  p.per = (int)per;
  p.chunks = (int)((HT + per - 1) / per);
  p.n_warps = tokens * p.chunks;
  const int64_t grid = (p.n_warps + AW - 1) / AW;
  if (grid > 0x7fffffff) return SSA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 g((unsigned)grid), t(32 * AW);
  if (d == 128) {
    if (interleaved) append_kernel<128, true><<<g, t, 0, st>>>(p);
    else append_kernel<128, false><<<g, t, 0, st>>>(p);
  } else {
    if (interleaved) append_kernel<64, true><<<g, t, 0, st>>>(p);
    else append_kernel<64, false><<<g, t, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? SSA_OK : SSA_ERR_CUDA;
}

int ssa_cache_evict(const void* k, const void* v, const float* mass, const int32_t* lens, void* k_out,
                    void* v_out, float* mass_out, int32_t* index_out, int32_t* lens_out, int B, int Hkv,
                    int cap, int cap_out, int d, int keep, int sink, int recent, void* stream) {
  using namespace ssa_cache;
  if (!k || !v || !mass || !lens || !k_out || !v_out || !mass_out || !index_out || !lens_out)
    return SSA_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || cap <= 0 || d <= 0 || keep <= 0 || sink < 0 || recent < 0) return SSA_ERR_INVALID_ARG;
  if ((int64_t)sink + recent > keep || cap_out < keep) return SSA_ERR_INVALID_ARG;
  if (mis(k, 16) || mis(v, 16) || mis(k_out, 16) || mis(v_out, 16) || mis(mass, 4) || mis(lens, 4) ||
      mis(mass_out, 4) || mis(index_out, 4) || mis(lens_out, 4))
    return SSA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSA_ERR_UNSUPPORTED;
  const size_t pairs = (size_t)B * Hkv;
  const int64_t rows = (int64_t)pairs * keep, per = (int64_t)GT / (d / 8) * GU;
  const int64_t grid = (rows + per - 1) / per;
  if (pairs > (1u << 24) || grid > 0x7fffffff || cap > (1 << 30)) return SSA_ERR_UNSUPPORTED;
  const ssa::Span span[9] = {
      {k_out, pairs * cap_out * d * 2}, {v_out, pairs * cap_out * d * 2}, {mass_out, pairs * cap_out * 4},
      {index_out, pairs * keep * 4},    {lens_out, (size_t)B * 4},        {k, pairs * cap * d * 2},
      {v, pairs * cap * d * 2},         {mass, pairs * cap * 4},          {lens, (size_t)B * 4}};
  for (int i = 0; i < 5; ++i)  // each output against every other tensor
    for (int j = i + 1; j < 9; ++j)
      if (ssa::overlap(span[i], span[j])) return SSA_ERR_INVALID_ARG;
  EvictParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.mass = mass;
  p.lens = lens;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.mass_out = mass_out;
  p.index_out = index_out;
  p.lens_out = lens_out;
  p.B = B;
  p.Hkv = Hkv;
  p.cap = cap;
  p.cap_out = cap_out;
  p.keep = keep;
  p.sink = sink;
  p.recent = recent;
  int sms = 0;
  if (sm_count(&sms) != SSA_OK) return SSA_ERR_CUDA;
  // blocks per (sequence, key head): as long as the GPU holds them at once and
  // a slice keeps a few keys for each of its 1024 threads
  int cs = 1;
  while (cs < 8 && pairs * cs * 2 <= (size_t)sms && cap / (cs * 2) >= 4 * ST) cs *= 2;
  const int slice = ((cap + cs - 1) / cs + 31) & ~31;
  p.max_keys = slice < MAX_KEYS ? slice : MAX_KEYS;
  const size_t smem = (size_t)p.max_keys * 4;
  if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_KEYS * 4) !=
      cudaSuccess)
    return SSA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(pairs * cs));
  cfg.blockDim = dim3(ST);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, p) != cudaSuccess) return SSA_ERR_CUDA;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(GT);
  cfg.dynamicSmemBytes = 0;
  return (d == 128 ? cudaLaunchKernelEx(&cfg, evict_gather_kernel<128>, p)
                   : cudaLaunchKernelEx(&cfg, evict_gather_kernel<64>, p)) == cudaSuccess
             ? SSA_OK
             : SSA_ERR_CUDA;
}

}  // extern "C"
