"""fp64 oracle of the key/value cache operators (include/ssa_cache.h), written
from their definitions, one head at a time, with no tiles and no running max.
Test infrastructure only.  Every function takes CPU tensors or arrays and
returns numpy arrays; the second result of the attention functions is what the
kernels' error bounds scale with."""
import numpy as np
import torch


def f64(x):
    return x.detach().to(torch.float64).cpu().numpy() if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)


def rotate(x, weight, pos, inv_freq, axis, interleaved, factor, eps):
    """Normalised and rotated rows of x [L, H, d]; pos [L, axes].  Second result: the size of each column's pair."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    size = np.abs(x)
    for p, f in enumerate(inv_freq):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + len(inv_freq))
        t = pos[:, axis[p]].astype(np.float64) * f
        c, s = factor * np.cos(t)[:, None], factor * np.sin(t)[:, None]
        ya, yb = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = np.hypot(ya, yb)
        x[..., a], x[..., b] = ya, yb
    return x, size


def tree_bits(mask, T):
    """[B, T, words] of 32 bits -> bool [B, T, T]."""
    w = np.ascontiguousarray(mask.cpu().numpy()).view(np.uint8)
    return np.unpackbits(w, axis=-1, bitorder="little")[..., :T].astype(bool)


def decode_tree(q, k, v, lens, mask, scale):
    """(out, lse, mean of |v| under the weights, largest sum of |q||k|), keys by the mask's bits."""
    qn, kn, vn = f64(q), f64(k), f64(v)
    B, T, Hq, d = qn.shape
    cap, Hkv = kn.shape[1:3]
    bits = tree_bits(mask, T)
    out, lse = np.zeros((B, T, Hq, d)), np.full((B, Hq, T), -np.inf)
    absv, dots = np.zeros((B, T, Hq, d)), np.zeros((B, Hq, T))
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            for i in range(T):
                draft = np.flatnonzero(bits[b, i])
                j = np.concatenate([np.arange(n), (n + draft)[n + draft < cap]])
                if len(j) == 0:
                    continue
                kk, vv = kn[b, j, hk], vn[b, j, hk]
                x = scale * (kk @ qn[b, i, h])
                m = x.max()
                w = np.exp(x - m)
                lse[b, h, i] = m + np.log(w.sum())
                w /= w.sum()
                out[b, i, h], absv[b, i, h] = w @ vv, w @ np.abs(vv)
                dots[b, h, i] = (np.abs(kk) @ np.abs(qn[b, i, h])).max()
    return out, lse, absv, dots


def attn_mass(q, k, lse, lens, causal, scale, window, mass, decay):
    """(mass [B, Hkv, cap], sum of weight * (|q||k| scale), sum of weight * (|score| + |lse| + 1))."""
    qn, kn, ln = f64(q), f64(k), f64(lse)
    B, Lq, Hq, d = qn.shape
    cap, Hkv = kn.shape[1:3]
    out, dots, args = (np.zeros((B, Hkv, cap)) for _ in range(3))
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        j = np.arange(n)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            for i in range(Lq - (window or Lq), Lq):
                if ln[b, h, i] == -np.inf:
                    continue
                see = j[j <= i + n - Lq] if causal else j
                x = scale * (kn[b, see, hk] @ qn[b, i, h])
                w = np.exp(x - ln[b, h, i])
                out[b, hk, see] += w
                dots[b, hk, see] += w * scale * (np.abs(kn[b, see, hk]) @ np.abs(qn[b, i, h]))
                args[b, hk, see] += w * (np.abs(x) + abs(ln[b, h, i]) + 1)
        if mass is not None:
            out[b, :, :n] += decay * f64(mass)[b, :, :n]
            args[b, :, :n] += decay * f64(mass)[b, :, :n]
    return out, dots, args


def evict_index(mass, n, keep, sink, recent):
    """The kept rows of one key head, ascending: python's sort by (-mass, index), NaN last."""
    if n <= keep:
        return list(range(n))
    mid = sorted(range(sink, n - recent), key=lambda j: (np.isnan(mass[j]), 0.0 if np.isnan(mass[j]) else -mass[j], j))
    return list(range(sink)) + sorted(mid[:keep - sink - recent]) + list(range(n - recent, n))
