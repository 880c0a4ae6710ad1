// sched.cuh -- even split of a batch of key/value caches of different lengths
// over the blocks of a grid, decided on the device from the lengths, and the
// bounded waits of the kernels that use it.
//
// The unit of work is one 128-key tile of one (sequence, inner index), inner
// = key head (and group of query rows).  Units are numbered sequence by
// sequence, inner index by inner index, tile by tile; block c of C takes the
// contiguous range [U c / C, U (c + 1) / C), so every block does the same number
// of tiles to within one whatever the lengths, and a range is a few segments,
// each a run of tiles of one (sequence, inner index).
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace ssa {

constexpr int MAX_SEQS = 1024;

struct Seg {
  int b, in;       // sequence, inner index
  int kt0, nt;     // key tiles [kt0, kt0 + nt)
  int tiles;       // tiles of the whole (sequence, inner index)
};

__device__ __forceinline__ int clamp_len(const int32_t* lens, int b, int cap) {
  return lens == nullptr ? cap : min(max(lens[b], 0), cap);
}

// pref[b] = tiles of sequences 0..b-1 (each counted once), pref[B] = all.  By one warp.
template <class Tiles>
__device__ __forceinline__ void tile_prefix(int* pref, int B, Tiles tiles) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    int x = b0 + lane < B ? tiles(b0 + lane) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += t;
    }
    if (b0 + lane < B) pref[b0 + lane + 1] = base + x;
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) pref[0] = 0;
}

// U c / C, rounded down, in 32 bits (C <= 2^15)
__device__ __forceinline__ int range_start(int U, int c, int C) { return U / C * c + U % C * c / C; }

// Walks one block's segments in order.  (The units of a batch fit 32 bits: its cache fits the GPU's memory.)
struct SegWalk {
  const int* pref;
  int inner, b, u, u1;
  __device__ __forceinline__ SegWalk(const int* pref_, int B, int inner_, int c, int C) : pref(pref_), inner(inner_) {
    const int U = inner * pref[B];
    if (C > U) C = U;
    u = c < C ? range_start(U, c, C) : U;
    u1 = c < C ? range_start(U, c + 1, C) : U;
    int lo = 0, hi = B - 1;  // the sequence that holds unit u
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (inner * pref[mid + 1] > u) hi = mid;
      else lo = mid + 1;
    }
    b = lo;
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (u >= u1) return false;
    while (inner * pref[b + 1] <= u) ++b;  // u < u1 <= U: some sequence holds it
    s.b = b;
    s.tiles = pref[b + 1] - pref[b];
    const int off = u - inner * pref[b];
    s.in = off / s.tiles;
    s.kt0 = off - s.in * s.tiles;
    s.nt = min(u1 - u, s.tiles - s.kt0);
    u += s.nt;
    return true;
  }
};

// Bounded wait that also gives up once another role of the block has: the
// first to run out of time raises the status word and the block's flag.
struct Waiter {
  volatile int* abort;
  int* status;
  unsigned long long limit_ns;  // at most 2^62
  __device__ __forceinline__ bool operator()(const uint64_t* bar, uint32_t parity) const {
    // Counted in clocks, two a nanosecond, more than the SM makes.  An attempt sleeps for as long as the hardware
    // likes, so a wait that has outlasted the limit gives up even where its attempt succeeded.
    const uint32_t a = smem_u32(bar);
    if (mbar_test_wait(a, parity)) return true;
    const unsigned long long t0 = clock64();
    for (;;) {
      const bool there = mbar_try_wait(a, parity);
      if (clock64() - t0 > 2 * limit_ns) {
        *abort = 1;
        atomicOr(status, 1);
        return false;
      }
      if (there) return true;
      if (*abort) return false;
    }
  }
};

}  // namespace ssa
