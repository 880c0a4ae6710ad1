"""ctypes binding of the key/value cache operators of libssa (include/ssa_cache.h).

``append``       normalise and rotate queries and keys, write keys and values into a cache
``decode_tree``  attention of drafted tokens (a tree, a chain, one token) over caches of different lengths
``attn_mass``    attention weight that each cached key received
``evict``        compaction of a cache to its heaviest keys

Marshalling and checks of what a C pointer cannot carry (dtype, device, layout);
every step runs in the CUDA kernels behind the C ABI and there is no fallback.
Functions that begin with ``ssa_`` are the C entry points and return their
status code; the others raise ``SSAError``.  Calls run on the device of the
tensors and on ``stream``, by default torch's current stream of that device;
outputs that are not passed in are allocated there.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
from typing import NamedTuple

import torch

from .ssa import SSA_ERR_INVALID_ARG, SSA_OK, SSAError, lib

EXPORTED = ["ssa_cache_append", "ssa_decode_tree", "ssa_decode_tree_workspace_bytes", "ssa_attn_mass",
            "ssa_cache_evict"]


def _bind():
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.ssa_cache_append.restype = I
    lib.ssa_cache_append.argtypes = [P, P, P, P, P, P, F, P, P, P, I, I, I, F, P, P, P, P, P] + [I] * 6 + [P]
    lib.ssa_decode_tree.restype = I
    lib.ssa_decode_tree.argtypes = [P] * 7 + [I] * 6 + [F, P, Z, P]
    lib.ssa_decode_tree_workspace_bytes.restype = Z
    lib.ssa_decode_tree_workspace_bytes.argtypes = [I] * 6
    lib.ssa_attn_mass.restype = I
    lib.ssa_attn_mass.argtypes = [P] * 6 + [I] * 8 + [F, F, P]
    lib.ssa_cache_evict.restype = I
    lib.ssa_cache_evict.argtypes = [P] * 9 + [I] * 8 + [P]


_bind()

ssa_cache_append = lib.ssa_cache_append
ssa_decode_tree = lib.ssa_decode_tree
ssa_decode_tree_workspace_bytes = lib.ssa_decode_tree_workspace_bytes
ssa_attn_mass = lib.ssa_attn_mass
ssa_cache_evict = lib.ssa_cache_evict


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise SSAError(SSA_ERR_INVALID_ARG, what)


def _refuse(name, dtype, shape, dev, contiguous=True):
    raise SSAError(SSA_ERR_INVALID_ARG, f"{name}: want {'contiguous ' if contiguous else ''}{dtype} {tuple(shape)} on "
                                        + ("the CPU" if dev < 0 else f"cuda:{dev}"))


# (The checks run on every call and cost as much as a small kernel: no text is put together unless one fails.)
def _tensor(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of this type and shape on device number ``dev`` (-1: the CPU)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        _refuse(name, dtype, shape, dev)
    return t.data_ptr()


def _optional(t, name, dtype, shape, dev):
    return None if t is None else _tensor(t, name, dtype, shape, dev)


def _heads(x, name):
    if not (isinstance(x, torch.Tensor) and x.dim() == 4 and x.dtype is torch.bfloat16 and x.is_cuda):
        raise SSAError(SSA_ERR_INVALID_ARG, f"{name}: want a 4-dimensional bf16 CUDA tensor")
    return x.shape


def _strided(x, name, shape, dev):
    """The batch, token and head stride of a tensor whose heads' columns are contiguous."""
    s = x.stride() if isinstance(x, torch.Tensor) else ()
    if not (s and x.dtype is torch.bfloat16 and x.shape == shape and x.get_device() == dev and s[3] == 1):
        _refuse(name + " (columns of a head contiguous)", torch.bfloat16, shape, dev, contiguous=False)
    return s[:3]


# (as torch's own generated code asks; the public calls build objects and cost as much as a launch)
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


class _On:
    """Makes the device of a call current, and a stream that the caller named; torch's allocations inside follow it."""

    __slots__ = ("dev", "stack")

    def __init__(self, dev, stream):
        self.dev, self.stack = dev, None
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=dev)
            _need(stream.device.index == dev, "stream: belongs to another device than the tensors")
        if stream is not None or _device() != dev:
            self.stack = contextlib.ExitStack()
            self.stack.enter_context(torch.cuda.device(dev))
            if stream is not None:
                self.stack.enter_context(torch.cuda.stream(stream))

    def __enter__(self):
        return _raw_stream(self.dev)

    def __exit__(self, *e):
        if self.stack is not None:
            self.stack.__exit__(*e)


def _done(status, what):
    if status != SSA_OK:
        raise SSAError(status, what)


def rope_frequencies(rot: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original: int = 8192, low: float = 1.0, high: float | None = None):
    """(inv_freq, factor) for ``append``: a CPU float64 tensor of rot / 2 radians per position, and what
    cosine and sine are multiplied by.

    ``scaling``: "none" base^(-2p / rot); "linear" all divided by ``factor``; "base" the base raised by
    factor^(rot / (rot - 2)), which divides the slowest by ``factor`` and leaves the fastest; "bands" by how often a
    pair turns within ``original`` positions: at most ``low`` turns divided by ``factor``, at least ``high`` (None: 4) left,
    between them a straight line between the two in turns; "ramp" the same with the line in the pair's number (``high``
    None: 32; the base above 1), and a factor of 1 + 0.1 ln(factor) on cosine and sine.
    """
    _need(rot > 0 and rot % 2 == 0 and base > 0 and factor > 0, "rope_frequencies: rot even, base and factor positive")
    n = rot // 2
    p = torch.arange(n, dtype=torch.float64)
    if scaling == "base":
        _need(rot > 2, "rope_frequencies: scaling 'base' needs rot > 2")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-p / n)
    if scaling in ("none", "base"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if high is None:
        high = 32.0 if scaling == "ramp" else 4.0
    _need(scaling in ("bands", "ramp") and 0 < low < high and original > 0,
          "rope_frequencies: scaling is none, linear, base, bands or ramp; 0 < low < high")
    _need(scaling == "bands" or base > 1, "rope_frequencies: scaling 'ramp' needs a base above 1")
    if scaling == "bands":
        turns = original * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        return f * (keep + (1 - keep) / factor), 1.0
    # the (whole) pair numbers that turn `high` and `low` times
    at = lambda t: n * math.log(original / (2 * math.pi * t)) / math.log(base)  # noqa: E731
    first, last = max(0, math.floor(at(high))), min(rot - 1, math.ceil(at(low)))
    keep = 1 - ((p - first) / max(last - first, 1e-3)).clamp(0, 1)
    return f * (keep + (1 - keep) / factor), (1.0 + 0.1 * math.log(factor) if factor > 1 else 1.0)


def append(q, k, v, k_cache, v_cache, positions=None, *, inv_freq=None, axis=None, interleaved=False, factor=1.0,
           q_weight=None, k_weight=None, eps=1e-6, start=None, count=None, out=None, stream=None):
    """Norm and rotation of q [B, L, Hq, d] and k [B, L, Hkv, d], and the write of k and v into rows
    start[b].. of k_cache, v_cache [B, cap, Hkv, d].  Returns the rotated queries [B, L, Hq, d].

    q, k, v may be strided (slices of one projection).  positions [B, L] or [B, L, axes] int32;
    inv_freq: CPU float64 [rot / 2] (None: no rotation); axis: CPU int32 [rot / 2]; weights fp32 [d];
    start, count int32 [B].  ``out`` (may be q): rows of tokens at and past count[b] keep what they hold;
    without ``out`` they are undefined.
    """
    B, L, Hq, d = _heads(q, "q")
    dev = q.get_device()
    Hkv = _heads(k, "k")[2]
    kv = (B, L, Hkv, d)
    strides = (ctypes.c_int64 * 9)(*_strided(q, "q", q.shape, dev), *_strided(k, "k", kv, dev),
                                   *_strided(v, "v", kv, dev))
    cap = _heads(k_cache, "k_cache")[1]
    kc = _tensor(k_cache, "k_cache", torch.bfloat16, (B, cap, Hkv, d), dev)
    vc = _tensor(v_cache, "v_cache", torch.bfloat16, (B, cap, Hkv, d), dev)
    rot, axes, freq, ax, pos = 0, 1, None, None, None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        freq = _tensor(inv_freq, "inv_freq", torch.float64, (rot // 2,), -1)
        _need(isinstance(positions, torch.Tensor) and positions.dim() in (2, 3), "positions: want [B, L] or [B, L, axes]")
        axes = positions.shape[2] if positions.dim() == 3 else 1
        pos = _tensor(positions, "positions", torch.int32, (B, L, axes) if positions.dim() == 3 else (B, L), dev)
        ax = _optional(axis, "axis", torch.int32, (rot // 2,), -1)
    wq = _optional(q_weight, "q_weight", torch.float32, (d,), dev)
    wk = _optional(k_weight, "k_weight", torch.float32, (d,), dev)
    s0 = _optional(start, "start", torch.int32, (B,), dev)
    cnt = _optional(count, "count", torch.int32, (B,), dev)
    with _On(dev, stream) as st:
        if out is None:
            out = torch.empty(B, L, Hq, d, dtype=torch.bfloat16, device=dev)
            qo = out.data_ptr()
        else:
            qo = _tensor(out, "out", torch.bfloat16, q.shape, dev)
        _done(ssa_cache_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, wq, wk, eps, pos, freq, ax, axes, rot,
                               int(interleaved), factor, s0, cnt, qo, kc, vc, B, L, Hq, Hkv, d, cap, st),
              "ssa_cache_append")
    return out


@functools.lru_cache(maxsize=256)
def _known_workspace(dev, B, T, Hq, Hkv, cap, d):
    n = ssa_decode_tree_workspace_bytes(B, T, Hq, Hkv, cap, d)
    if n == 0:
        raise LookupError  # (not kept)
    return n


def _tree_workspace(*shape):
    try:
        return _known_workspace(*shape)
    except LookupError:
        return 16  # a shape that the call itself refuses


def decode_tree(q, k, v, lens, tree_mask, *, scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of T drafted tokens per sequence (q [B, T, Hq, d]) over its cache k, v [B, cap, Hkv, d]:
    the keys before lens[b], and draft key t (row lens[b] + t) where bit t of tree_mask[b, i] is set.

    lens int32 [B]; tree_mask int32 or uint32 [B, T, ceil(T / 32)].  Returns (out [B, T, Hq, d] bf16,
    lse [B, Hq, T] fp32).  ``workspace``: uint8, ``ssa_decode_tree_workspace_bytes`` bytes.
    """
    B, T, Hq, d = _heads(q, "q")
    dev = q.get_device()
    _, cap, Hkv, _ = _heads(k, "k")
    qp = _tensor(q, "q", torch.bfloat16, q.shape, dev)
    kp = _tensor(k, "k", torch.bfloat16, (B, cap, Hkv, d), dev)
    vp = _tensor(v, "v", torch.bfloat16, (B, cap, Hkv, d), dev)
    lp = _tensor(lens, "lens", torch.int32, (B,), dev)
    words = (B, T, (T + 31) // 32)
    mp = _tensor(tree_mask, "tree_mask",
                 torch.uint32 if getattr(tree_mask, "dtype", None) == torch.uint32 else torch.int32, words, dev)
    if scale is None:
        scale = d ** -0.5
    with _On(dev, stream) as st:
        if out is None:
            out = torch.empty_like(q)
            op = out.data_ptr()
        else:
            op = _tensor(out, "out", torch.bfloat16, q.shape, dev)
        if lse is None:
            lse = torch.empty(B, Hq, T, dtype=torch.float32, device=dev)
            sp = lse.data_ptr()
        else:
            sp = _tensor(lse, "lse", torch.float32, (B, Hq, T), dev)
        if workspace is None:
            workspace = torch.empty(_tree_workspace(dev, B, T, Hq, Hkv, cap, d), dtype=torch.uint8, device=dev)
        elif not (isinstance(workspace, torch.Tensor) and workspace.get_device() == dev and workspace.is_contiguous()):
            raise SSAError(SSA_ERR_INVALID_ARG, f"workspace: want a contiguous tensor on cuda:{dev}")
        _done(ssa_decode_tree(qp, kp, vp, op, sp, lp, mp, B, T, Hq, Hkv, cap, d, scale, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), st), "ssa_decode_tree")
    return out, lse


def attn_mass(q, k, lse, *, lens=None, causal=True, scale=None, window=0, mass=None, decay=1.0, out=None, stream=None):
    """Attention weight that each key of k [B, cap, Hkv, d] received from the rows q [B, Lq, Hq, d] (the last
    ``window`` of them; 0: all), given their lse [B, Hq, Lq] from the attention: decay * mass + the sum over rows and
    the query heads of a key head.  Returns mass [B, Hkv, cap] fp32 (``out``; may be ``mass`` itself), 0 past lens[b].

    The weights of dense attention: every key at or before a row (position i + lens[b] - Lq) counts, whether or not the
    attention looked at it.  Rows padded on the right: lens start[b] + Lq, and a lse of -inf in the padding's rows.
    """
    B, Lq, Hq, d = _heads(q, "q")
    dev = q.get_device()
    _, cap, Hkv, _ = _heads(k, "k")
    qp = _tensor(q, "q", torch.bfloat16, q.shape, dev)
    kp = _tensor(k, "k", torch.bfloat16, (B, cap, Hkv, d), dev)
    sp = _tensor(lse, "lse", torch.float32, (B, Hq, Lq), dev)
    lp = _optional(lens, "lens", torch.int32, (B,), dev)
    mp = _optional(mass, "mass", torch.float32, (B, Hkv, cap), dev)
    _need(0 <= window <= Lq, "window: want 0 (all rows) to Lq")
    if scale is None:
        scale = d ** -0.5
    with _On(dev, stream) as st:
        if out is None:
            out = torch.empty(B, Hkv, cap, dtype=torch.float32, device=dev)
            op = out.data_ptr()
        else:
            op = _tensor(out, "out", torch.float32, (B, Hkv, cap), dev)
        _done(ssa_attn_mass(qp, kp, sp, lp, mp, op, B, Lq, window, Hq, Hkv, cap, d, int(causal), scale, decay, st),
              "ssa_attn_mass")
    return out


class Evicted(NamedTuple):
    k: torch.Tensor        # [B, cap_out, Hkv, d]
    v: torch.Tensor
    mass: torch.Tensor     # [B, Hkv, cap_out]
    index: torch.Tensor    # [B, Hkv, keep] int32, -1 past the kept
    lens: torch.Tensor     # [B] int32


def evict(k, v, mass, lens, *, keep, sink=0, recent=0, k_out=None, v_out=None, mass_out=None, index=None, new_lens=None,
          stream=None):
    """Compact caches k, v [B, cap, Hkv, d] to at most ``keep`` keys a key head: the first ``sink``, the last
    ``recent`` and the heaviest by mass [B, Hkv, cap] of the rest, in ascending order.  k_out, v_out
    [B, cap_out, Hkv, d] with cap_out >= keep (default keep); their rows past the kept ones keep what they hold.
    Returns ``Evicted``.
    """
    B, cap, Hkv, d = _heads(k, "k")
    dev = k.get_device()
    kp = _tensor(k, "k", torch.bfloat16, k.shape, dev)
    vp = _tensor(v, "v", torch.bfloat16, k.shape, dev)
    mp = _tensor(mass, "mass", torch.float32, (B, Hkv, cap), dev)
    lp = _tensor(lens, "lens", torch.int32, (B,), dev)
    _need(1 <= keep < 2 ** 31 and sink >= 0 and recent >= 0 and sink + recent <= keep, "keep, sink, recent: want sink + recent <= keep")
    with _On(dev, stream) as st:
        cap_out = keep
        for t, name in ((k_out, "k_out"), (v_out, "v_out")):
            if t is not None:
                cap_out = _heads(t, name)[1]

        def output(t, name, dtype, *shape):
            if t is None:
                t = torch.empty(shape, dtype=dtype, device=dev)
                return t, t.data_ptr()
            return t, _tensor(t, name, dtype, shape, dev)

        k_out, ko = output(k_out, "k_out", torch.bfloat16, B, cap_out, Hkv, d)
        v_out, vo = output(v_out, "v_out", torch.bfloat16, B, cap_out, Hkv, d)
        mass_out, mo = output(mass_out, "mass_out", torch.float32, B, Hkv, cap_out)
        index, io = output(index, "index", torch.int32, B, Hkv, keep)
        new_lens, lo = output(new_lens, "new_lens", torch.int32, B)
        _done(ssa_cache_evict(kp, vp, mp, lp, ko, vo, mo, io, lo, B, Hkv, cap, cap_out, d, keep, sink, recent, st),
              "ssa_cache_evict")
    return Evicted(k_out, v_out, mass_out, index, new_lens)
