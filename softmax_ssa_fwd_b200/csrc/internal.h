// internal.h -- host helpers shared by the kernels of libssa (not part of
// the C ABI).
#pragma once
#include <cuda.h>

#include <cstddef>
#include <cstdint>

namespace ssa {

// [B, L, H, d] bf16 -> 4-D TMA tensor map (d, H, L, B) with a (64, 1, rows, 1)
// box and 128-byte swizzle; coordinates past the tensor read zeros.
bool tma_map_bf16(CUtensorMap* map, const void* base, int B, int L, int H, int d, int rows);
// The same with a (64, heads, rows, 1) box: `heads` neighbouring heads of each
// of `rows` tokens land as rows * heads consecutive tile rows, token-major.
bool tma_map_bf16_box(CUtensorMap* map, const void* base, int B, int L, int H, int d, int heads, int rows);

// Memory of a tensor, for refusing outputs that lie over something else of the call.
struct Span {
  const void* at;
  size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && x < y + b.bytes && y < x + a.bytes;
}

// The per-device status word that a timed-out bounded device wait raises
// (ssa_device_status reads and clears it); nullptr on failure.
int* device_status_word(int dev);

// The current limit of one device-side wait (ssa_set_wait_timeout_ns), at most
// 2^62, a century, so that a kernel can count it in half nanoseconds.
unsigned long long wait_timeout_ns();

}  // namespace ssa
