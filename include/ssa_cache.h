/*
 * ssa_cache.h -- C ABI of the key/value cache operators of libssa (NVIDIA
 * B200, sm_100a): writing a cache (per-head norm, position rotation, append),
 * attention of drafted tokens over caches of different lengths, the attention
 * weight each cached key received, and the compaction of a cache to its
 * heaviest keys.  They stand beside ssa_fwd and ssa_decode of ssa.h and share
 * its conventions:
 *   - tensor pointers are DEVICE pointers on the current CUDA device, owned by
 *     the caller; bf16 tensors 16-byte aligned, 32-bit arrays 4-byte aligned
 *     (SSA_ERR_INVALID_ARG otherwise).  Pointers marked HOST are read during
 *     the call and not kept.
 *   - a cache is two tensors k, v [B, cap, Hkv, d] bf16, contiguous: row j of
 *     sequence b is its j-th cached token, and rows at and past the sequence's
 *     length hold anything (NaN included) without touching a result.
 *     q is [B, L, Hq, d]; query head hq reads key head hq / (Hq / Hkv).
 *   - lens [B] int32 is DEVICE memory: lengths are read by the kernels, so a
 *     captured graph replays with the lengths of the moment.  A length outside
 *     [0, cap] counts as the nearest of the two.
 *   - d in {64, 128}.
 *   - Work is enqueued on `stream`; argument errors are reported at once with
 *     the status codes of ssa.h and nothing is enqueued.  No exception crosses
 *     this boundary, and no entry point synchronises.  The first call of
 *     ssa_decode_tree or ssa_attn_mass on a device allocates the 4-byte status
 *     word that ssa_device_status reads: make it (or any ssa_fwd / ssa_decode
 *     call) before capturing a graph.
 *   - An output must not lie over an input, over the workspace or over another
 *     output (SSA_ERR_INVALID_ARG), but for the two cases named below.
 *   - Results do not depend on the order in which blocks run: the same call
 *     on the same GPU gives the same bits.
 */
#ifndef SSA_CACHE_H
#define SSA_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "ssa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Normalise, rotate and append.  For every token i < count[b] of sequence b and
 * every head of q and k
 *     y_c = x_c * rsqrt(mean(x^2) + eps) * weight_c          (weight given; fp32)
 *     (y_a, y_b) <- factor * (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
 * for the rot / 2 pairs (a, b) of the head's first `rot` columns,
 * t = positions[b, i, axis[p]] * inv_freq[p] for pair p; the other columns are
 * not rotated and not scaled by factor.  Pair p is columns (p, p + rot / 2), or
 * (2p, 2p + 1) when `interleaved`.  The rotated q goes to q_out, the rotated k
 * and the unchanged v to cache row start[b] + i.  All arithmetic is in fp32 and
 * rounded to bf16 once; angles are reduced exactly, so far positions lose nothing.
 *   q, k, v:   bf16 [B, L, H, d] in any layout with contiguous heads' columns:
 *              strides[9] (HOST, in elements) holds the batch, token and head
 *              stride of q, then of k, then of v.  Each a non-negative multiple
 *              of 8, pointers 16-byte aligned (a slice of a fused projection works).
 *   q_weight, k_weight: fp32 [d], or NULL for no norm of that tensor.
 *   positions: int32 [B, L, axes] (NULL allowed when rot == 0).
 *   inv_freq:  HOST, double [rot / 2], radians per position, finite.
 *   axis:      HOST, int32 [rot / 2], each in [0, axes), or NULL for all 0.
 *   start:     int32 [B], NULL for 0.  A cache row outside [0, cap) is not
 *              written (q_out is).
 *   count:     int32 [B], NULL for L: tokens of sequence b in this padded batch.
 *              Tokens at and past count[b] change nothing: their q_out rows and
 *              cache rows keep what they hold.
 *   q_out:     bf16 [B, L, Hq, d] contiguous; may be q itself when q is contiguous.
 *   Limits: rot a multiple of 16, 0 <= rot <= d; 1 <= axes <= 4
 *   (SSA_ERR_UNSUPPORTED otherwise). */
int ssa_cache_append(const void* q, const void* k, const void* v, const int64_t* strides,
                     const float* q_weight, const float* k_weight, float eps,
                     const int32_t* positions, const double* inv_freq, const int32_t* axis, int axes,
                     int rot, int interleaved, float factor, const int32_t* start,
                     const int32_t* count, void* q_out, void* k_cache, void* v_cache, int B, int L,
                     int Hq, int Hkv, int d, int cap, void* stream);

/* Attention of T drafted tokens per sequence over its cache: row i of sequence
 * b sees every cached key j < lens[b], and draft key t (cache row lens[b] + t,
 * appended before the call) iff bit t % 32 of word t / 32 of tree_mask[b, i] is set.
 * A tree's row holds its ancestors' bits and its own; a chain is the lower
 * triangle; T = 1 with bit 0 set is a decode step over sequences of different
 * lengths.  out = softmax(scale * q.k) v over the seen keys, lse its natural
 * log-sum-exp; a row that sees nothing gets out = 0 and lse = -inf.  Dense: no
 * key tile is skipped.  Draft rows at and past cap do not exist; bits at and past
 * T are ignored.  A key that a row does not see has no influence on it, whatever
 * it holds.  As in ssa_fwd and ssa_decode, the weights are rounded to bf16 for
 * their product with V (a relative error of at most 2^-8 each), and their
 * sum is of the unrounded ones; scores, maxima, sums and accumulators are fp32.
 *   q, out:    bf16 [B, T, Hq, d];  lse: fp32 [B, Hq, T]
 *   lens:      int32 [B]: cached keys before the draft
 *   tree_mask: uint32 [B, T, ceil(T / 32)]
 *   workspace: device scratch, 16-byte aligned, at least
 *              ssa_decode_tree_workspace_bytes() bytes, used by this call only
 *              while it runs (calls that may overlap need one each).
 *   Limits: T <= 128, Hq / Hkv <= 128, B <= 1024 (SSA_ERR_UNSUPPORTED otherwise). */
int ssa_decode_tree(const void* q, const void* k, const void* v, void* out, float* lse,
                    const int32_t* lens, const uint32_t* tree_mask, int B, int T, int Hq, int Hkv,
                    int cap, int d, float scale, void* workspace, size_t workspace_bytes,
                    void* stream);

/* Bytes of workspace ssa_decode_tree needs for this shape on the current device
 * (0 for invalid or unsupported sizes, or without a device). */
size_t ssa_decode_tree_workspace_bytes(int B, int T, int Hq, int Hkv, int cap, int d);

/* Attention weight that each cached key received:
 *     mass_out[b, h, j] = decay * mass_in[b, h, j]
 *                       + sum over rows i and the query heads g of key head h of
 *                         exp(scale * q[b, i, g] . k[b, j, h] - lse[b, g, i])
 * for j < lens[b], and 0 for j in [lens[b], cap).  lse is what ssa_fwd,
 * ssa_decode or ssa_decode_tree returned for these rows.  Only the last
 * `window` of the Lq rows count (0: all).  causal != 0: row i sits at position
 * i + lens[b] - Lq and gives weight to keys at and before it.  A row whose lse is
 * -inf gives none; a lse of NaN makes the keys that its row sees NaN, and no others.
 * Every key at or before a row counts, whether or not the attention looked at it:
 * the weights are those of dense attention.  With the lse of a skip, N:M or
 * block-mask call, or of a tree's row and branches that it does not see, they sum
 * to more than 1.
 * Rows padded on the right (ssa_cache_append with count[b] < L): give the length
 * start[b] + L (at most cap), so that row i sits at start[b] + i, and a lse of -inf
 * in the padding's rows; choose the rows that count by their lse then, not by
 * `window`, and hold 0 in mass_in for the padding's keys.
 *   q: bf16 [B, Lq, Hq, d];  k: bf16 [B, cap, Hkv, d];  lse: fp32 [B, Hq, Lq]
 *   lens: int32 [B], NULL for cap
 *   mass_in, mass_out: fp32 [B, Hkv, cap]; mass_in NULL counts as 0 (decay is
 *   then not used); mass_out may be mass_in.  decay finite, >= 0.
 *   Limits: B <= 1024, Hq / Hkv <= 128 (SSA_ERR_UNSUPPORTED otherwise). */
int ssa_attn_mass(const void* q, const void* k, const float* lse, const int32_t* lens,
                  const float* mass_in, float* mass_out, int B, int Lq, int window, int Hq, int Hkv,
                  int cap, int d, int causal, float scale, float decay, void* stream);

/* Compact each sequence's cache to at most `keep` keys, per key head.  With
 * n = lens[b] <= keep every key stays.  Otherwise the first `sink`, the last
 * `recent` and, of the keys between, the keep - sink - recent with the largest
 * mass stay (ties go to the lower index; NaN ranks below every number), in
 * ascending order.
 *   k, v:         bf16 [B, cap, Hkv, d];  mass: fp32 [B, Hkv, cap]
 *   k_out, v_out: bf16 [B, cap_out, Hkv, d], cap_out >= keep; rows past the kept
 *                 ones keep what they hold.
 *   mass_out:     fp32 [B, Hkv, cap_out]: the kept masses, 0 past them.
 *   index_out:    int32 [B, Hkv, keep]: the kept rows of k, -1 past them.
 *   lens_out:     int32 [B]: min(lens[b], keep).
 *   keep >= 1, sink >= 0, recent >= 0, sink + recent <= keep. */
int ssa_cache_evict(const void* k, const void* v, const float* mass, const int32_t* lens,
                    void* k_out, void* v_out, float* mass_out, int32_t* index_out,
                    int32_t* lens_out, int B, int Hkv, int cap, int cap_out, int d, int keep,
                    int sink, int recent, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSA_CACHE_H */
