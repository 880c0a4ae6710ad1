"""Host-side checks of the key/value cache operators (no GPU needed): the
library exports what include/ssa_cache.h declares and refuses bad arguments
before touching CUDA; the Python calls refuse what a pointer cannot carry; the
frequency helper; pins of the fp64 oracle (oracle/cache.py) against torch's
own fp64 attention, complex rotations and sorting."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import cache as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssa_cache.h")


@pytest.fixture(scope="module")
def cache():
    from softmax_ssa_fwd_b200 import build
    build.build()
    from softmax_ssa_fwd_b200 import cache as mod
    return mod


def test_library_exports_what_the_header_declares(cache):
    from softmax_ssa_fwd_b200 import ssa
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ssa_[a-z_]+)\s*\(", text)))
    assert names == sorted(cache.EXPORTED)
    lib = ctypes.CDLL(ssa.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)


# ------------------------------------------------------------------ refusals

def _append(cache, **over):
    a = dict(q=0x10000, k=0x20000, v=0x30000, wq=0x40000, wk=0x41000, eps=1e-6, pos=0x50000, axes=1, rot=128,
             pairs=0, factor=1.0, start=0x60000, count=0x61000, out=0x70000, kc=0x80000, vc=0x90000, B=2, L=3, Hq=4,
             Hkv=2, d=128, cap=16, axis=None, strides=[1536, 512, 128, 768, 256, 128, 768, 256, 128])
    a["freq"] = [0.1] * 96
    a.update(over)
    c = lambda t, v: None if v is None else (t * len(v))(*v)  # noqa: E731
    return cache.ssa_cache_append(a["q"], a["k"], a["v"], c(ctypes.c_int64, a["strides"]), a["wq"], a["wk"], a["eps"],
                                  a["pos"], c(ctypes.c_double, a["freq"]), c(ctypes.c_int32, a["axis"]), a["axes"],
                                  a["rot"], a["pairs"], a["factor"], a["start"], a["count"], a["out"], a["kc"], a["vc"],
                                  a["B"], a["L"], a["Hq"], a["Hkv"], a["d"], a["cap"], None)


@pytest.mark.parametrize("over", [
    dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(kc=0), dict(vc=0), dict(pos=0), dict(freq=None),
    dict(strides=None), dict(B=0), dict(L=0), dict(Hq=0), dict(Hkv=-1), dict(d=0), dict(cap=0), dict(rot=-16),
    dict(q=0x10008), dict(kc=0x80004), dict(out=0x70002), dict(wq=0x40002), dict(pos=0x50001), dict(count=0x61002),
    dict(start=0x60003), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(factor=math.nan),
])
def test_append_invalid(cache, over):
    assert _append(cache, **over) == -1


def test_append_invalid_host_arrays(cache):
    assert _append(cache, strides=[1536, 512, 128, 768, 256, 128, 768, 260, 128]) == -1
    assert _append(cache, strides=[1536, 512, 128, 768, 256, 128, -768, 256, 128]) == -1
    assert _append(cache, freq=[0.1] * 63 + [math.inf]) == -1
    assert _append(cache, axes=2, axis=[0] * 63 + [2]) == -1
    assert _append(cache, axes=2, axis=[-1] + [0] * 63) == -1


@pytest.mark.parametrize("over", [
    dict(kc=0x10000), dict(vc=0x20000 + 0x400), dict(vc=0x80000), dict(kc=0x70000), dict(out=0x20000), dict(out=0x30000),
    dict(out=0x10000 + 0x100), dict(out=0x10000, strides=[1664, 544, 136, 768, 256, 128, 768, 256, 128]),
])
def test_append_outputs_over_other_tensors(cache, over):
    assert _append(cache, **over) == -1


@pytest.mark.parametrize("out", ["out", "kc", "vc"])
@pytest.mark.parametrize("what", ["wq", "wk", "pos", "start", "count"])
def test_append_outputs_over_small_inputs(cache, out, what):
    base = dict(out=0x70000, kc=0x80000, vc=0x90000)[out]
    assert _append(cache, **{what: base}) == _append(cache, **{what: base + 0x400}) == -1
    if not torch.cuda.is_available():  # right behind it, or not read: on to CUDA, which is not there
        behind = base + (2 * 3 * 4 * 128 * 2 if out == "out" else 2 * 16 * 2 * 128 * 2)
        assert _append(cache, **{what: behind}) == -3
        if what == "pos":
            assert _append(cache, pos=base, rot=0) == -3


def test_append_over_its_own_queries_is_allowed(cache):
    if torch.cuda.is_available():
        pytest.skip("needs the no-GPU path")
    assert _append(cache) == _append(cache, out=0x10000) == -3  # on to CUDA, which is not there


@pytest.mark.parametrize("over", [dict(d=96, rot=0), dict(rot=24), dict(rot=144), dict(axes=0), dict(axes=5),
                                  dict(d=64)])
def test_append_unsupported(cache, over):
    assert _append(cache, **over) == -2


def _tree(cache, **over):
    a = dict(q=0x10000000, k=0x20000000, v=0x30000000, out=0x40000000, lse=0x50000000, lens=0x60000000, mask=0x70000000,
             B=2, T=4, Hq=8, Hkv=2, cap=300, d=128, scale=0.1, ws=0x80000000, wsb=1 << 30)
    a.update(over)
    return cache.ssa_decode_tree(*a.values(), None)


@pytest.mark.parametrize("over", [
    dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(lse=0), dict(lens=0), dict(mask=0), dict(ws=0), dict(B=0),
    dict(T=0), dict(Hq=0), dict(Hkv=0), dict(cap=0), dict(d=-64), dict(Hq=7), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=math.nan), dict(scale=math.inf), dict(q=0x10000008), dict(v=0x30000002), dict(ws=0x80000004), dict(lse=0x50000002),
    dict(lens=0x60000001), dict(mask=0x70000002),
    dict(out=0x10000000), dict(out=0x20000000), dict(lse=0x10000040), dict(ws=0x30000000), dict(lse=0x60000000),
    dict(out=0x50000000 - 0x1000), dict(ws=0x40000000, wsb=1 << 30),
])
def test_tree_invalid(cache, over):
    assert _tree(cache, **over) == -1


@pytest.mark.parametrize("over", [dict(T=129), dict(Hq=258, Hkv=2), dict(B=1025), dict(d=96), dict(d=256)])
def test_tree_unsupported(cache, over):
    assert _tree(cache, **over) == -2
    a = dict(B=2, T=4, Hq=8, Hkv=2, cap=300, d=128)
    a.update(over)
    assert cache.ssa_decode_tree_workspace_bytes(*a.values()) == 0


def _mass(cache, **over):
    a = dict(q=0x10000000, k=0x20000000, lse=0x30000000, lens=0x40000000, min=0x50000000, out=0x60000000, B=2, Lq=4, window=0, Hq=8, Hkv=2,
             cap=300, d=128, causal=1, scale=0.1, decay=0.5)
    a.update(over)
    return cache.ssa_attn_mass(*a.values(), None)


@pytest.mark.parametrize("over", [
    dict(q=0), dict(k=0), dict(lse=0), dict(out=0), dict(B=0), dict(Lq=0), dict(window=-1), dict(window=5), dict(Hq=0),
    dict(Hkv=0), dict(Hq=9), dict(cap=0), dict(d=0), dict(scale=0.0), dict(scale=math.inf), dict(decay=-0.1),
    dict(decay=math.nan), dict(decay=math.inf), dict(q=0x10000004), dict(k=0x20000008), dict(lse=0x30000002),
    dict(min=0x50000001), dict(out=0x60000002), dict(lens=0x40000002), dict(out=0x10000000), dict(out=0x20000000),
    dict(out=0x30000000), dict(out=0x40000000), dict(out=0x50000004),
])
def test_mass_invalid(cache, over):
    assert _mass(cache, **over) == -1


@pytest.mark.parametrize("over", [dict(d=32), dict(B=1025), dict(Hq=258)])
def test_mass_unsupported(cache, over):
    assert _mass(cache, **over) == -2


def _evict(cache, **over):
    a = dict(k=0x10000000, v=0x20000000, mass=0x30000000, lens=0x31000000, ko=0x40000000, vo=0x50000000, mo=0x60000000,
             io=0x61000000, lo=0x62000000, B=2, Hkv=2, cap=1000, cap_out=120, d=128, keep=100, sink=4, recent=10)
    a.update(over)
    return cache.ssa_cache_evict(*a.values(), None)


@pytest.mark.parametrize("over", [
    dict(k=0), dict(v=0), dict(mass=0), dict(lens=0), dict(ko=0), dict(vo=0), dict(mo=0), dict(io=0), dict(lo=0),
    dict(B=0), dict(Hkv=0), dict(cap=0), dict(d=0), dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=91),
    dict(cap_out=99), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(k=0x10000008), dict(vo=0x50000002),
    dict(mass=0x30000002), dict(io=0x61000001), dict(lo=0x62000002),
    dict(ko=0x10000000), dict(vo=0x10000000 + 2 * 2 * 1000 * 256 - 16), dict(vo=0x40000000), dict(mo=0x30000000),
    dict(lo=0x31000000), dict(io=0x60000000 + 4), dict(lo=0x61000000 + 400),
])
def test_evict_invalid(cache, over):
    assert _evict(cache, **over) == -1


@pytest.mark.parametrize("over", [dict(d=96), dict(B=1 << 24, Hkv=2)])
def test_evict_unsupported(cache, over):
    assert _evict(cache, **over) == -2


def test_python_calls_refuse_other_tensors(cache):
    from softmax_ssa_fwd_b200 import ssa
    t = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: cache.append(t, t, t, t, t), lambda: cache.decode_tree(t, t, t, i, i),
                 lambda: cache.attn_mass(t, t, t), lambda: cache.evict(t, t, t, i, keep=1)):
        with pytest.raises(ssa.SSAError) as e:
            call()
        assert e.value.status == ssa.SSA_ERR_INVALID_ARG and "CUDA tensor" in str(e.value)


# ------------------------------------------------------------------ frequencies

def test_rope_frequencies(cache):
    rot, base = 64, 10000.0
    plain = [base ** (-2 * p / rot) for p in range(rot // 2)]
    f, a = cache.rope_frequencies(rot, base)
    assert f.dtype == torch.float64 and a == 1.0 and np.allclose(f, plain, rtol=1e-14)
    f, _ = cache.rope_frequencies(rot, base, scaling="linear", factor=4.0)
    assert np.allclose(f, np.array(plain) / 4, rtol=1e-14)
    f, _ = cache.rope_frequencies(rot, base, scaling="base", factor=4.0)
    assert f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 4, rel_tol=1e-12)
    f, a = cache.rope_frequencies(rot, base, scaling="bands", factor=8.0, original=8192)
    assert a == 1.0
    for p in range(rot // 2):
        turns = 8192 * plain[p] / (2 * math.pi)
        keep = min(max((turns - 1) / 3, 0), 1)
        assert math.isclose(f[p], plain[p] * (keep + (1 - keep) / 8), rel_tol=1e-12)
    f, a = cache.rope_frequencies(rot, base, scaling="ramp", factor=16.0, original=4096, low=1.0, high=32.0)
    assert math.isclose(a, 0.1 * math.log(16) + 1) and f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 16)
    r = f.numpy() / plain
    assert (np.diff(r) <= 1e-12).all()


def test_rope_frequencies_defaults_of_each_scaling(cache):
    for scaling, high in (("bands", 4.0), ("ramp", 32.0)):
        got = cache.rope_frequencies(64, scaling=scaling, factor=16.0, original=4096)
        want = cache.rope_frequencies(64, scaling=scaling, factor=16.0, original=4096, low=1.0, high=high)
        other = cache.rope_frequencies(64, scaling=scaling, factor=16.0, original=4096, low=1.0, high=36.0 - high)
        assert torch.equal(got[0], want[0]) and got[1] == want[1] and not torch.equal(got[0], other[0])


@pytest.mark.parametrize("base", [1.0, 0.5])
def test_rope_frequencies_ramp_needs_falling_frequencies(cache, base):
    from softmax_ssa_fwd_b200 import ssa
    with pytest.raises(ssa.SSAError) as e:
        cache.rope_frequencies(64, base, scaling="ramp", factor=2.0)
    assert e.value.status == ssa.SSA_ERR_INVALID_ARG


def test_rope_frequencies_refusals(cache):
    from softmax_ssa_fwd_b200 import ssa
    for kw in (dict(rot=0), dict(rot=7), dict(rot=64, base=0.0), dict(rot=64, factor=0.0), dict(rot=64, scaling="other"),
               dict(rot=64, scaling="bands", low=4.0, high=1.0), dict(rot=2, scaling="base"),
               dict(rot=64, scaling="ramp", original=0)):
        with pytest.raises(ssa.SSAError):
            cache.rope_frequencies(**kw)


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("pairs", [False, True])
def test_oracle_rotation_is_a_complex_product(pairs):
    L, H, d, rot = 5, 3, 16, 12
    g = torch.Generator().manual_seed(1)
    x = torch.randn(L, H, d, generator=g, dtype=torch.float64)
    w = torch.randn(d, generator=g, dtype=torch.float64)
    pos, freq = torch.randint(0, 99, (L, 2), generator=g), torch.rand(rot // 2, generator=g, dtype=torch.float64)
    axis = [0, 1, 1, 0, 1, 0]
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w
    a = y[..., 0:rot:2] if pairs else y[..., :rot // 2]
    b = y[..., 1:rot:2] if pairs else y[..., rot // 2:rot]
    t = pos[:, axis].double() * freq
    z = torch.complex(a, b) * torch.polar(torch.full_like(t, 1.5), t)[:, None]
    y[..., :rot] = torch.stack([z.real, z.imag], -1).flatten(-2) if pairs else torch.cat([z.real, z.imag], -1)
    got, size = oracle.rotate(x.numpy(), w.numpy(), pos.numpy(), freq.numpy(), axis, pairs, 1.5, 1e-5)
    assert np.allclose(got, y, atol=1e-12) and (size + 1e-12 >= np.abs(got)).all()


def test_oracle_tree_is_masked_attention():
    B, T, Hq, Hkv, d, cap = 2, 37, 4, 2, 16, 60
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(B, n, h, d, generator=g, dtype=torch.float64) for n, h in ((T, Hq), (cap, Hkv), (cap, Hkv)))
    bits = torch.rand(B, T, 64, generator=g) < 0.4
    mask = torch.from_numpy(np.packbits(bits.numpy(), axis=-1, bitorder="little").view(np.int32))
    lens = torch.tensor([20, 30])  # the second draft runs past the cache
    out, lse, _, _ = oracle.decode_tree(q, k, v, lens, mask, 0.25)
    for b in range(B):
        n = int(lens[b])
        see = torch.zeros(T, cap, dtype=torch.bool)
        see[:, :n] = True
        m = min(T, cap - n)
        see[:, n:n + m] = bits[b, :, :m]
        want = torch.nn.functional.scaled_dot_product_attention(
            q[b].transpose(0, 1), k[b].transpose(0, 1).repeat_interleave(2, 0),
            v[b].transpose(0, 1).repeat_interleave(2, 0), attn_mask=see, scale=0.25)
        assert np.allclose(out[b], want.transpose(0, 1), atol=1e-12)
        x = torch.einsum("thd,jhd->htj", q[b], k[b].repeat_interleave(2, 1)) * 0.25
        assert np.allclose(lse[b], torch.logsumexp(x.masked_fill(~see, -math.inf), -1), atol=1e-12)


def test_oracle_mass_is_a_column_sum():
    B, Lq, Hq, Hkv, d, cap = 2, 9, 4, 2, 16, 40
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(B, n, h, d, generator=g, dtype=torch.float64) for n, h in ((Lq, Hq), (cap, Hkv)))
    lens = torch.tensor([33, 12])
    x = torch.einsum("bihd,bjhd->bhij", q, k.repeat_interleave(2, 2)) * 0.25
    see = torch.arange(cap)[None, None] <= torch.arange(Lq)[None, :, None] + lens[:, None, None] - Lq
    x = x.masked_fill(~see[:, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    old = torch.rand(B, Hkv, cap, generator=g, dtype=torch.float64)
    got, _, _ = oracle.attn_mass(q, k, lse, lens, True, 0.25, 4, old, 0.5)
    want = torch.softmax(x, -1)[:, :, -4:].sum(2).view(B, Hkv, 2, cap).sum(2)
    live = torch.arange(cap)[None, None] < lens[:, None, None]
    want = (want + 0.5 * old).masked_fill(~live, 0.0)
    assert np.allclose(got, want, atol=1e-12)


def test_oracle_eviction_order():
    nan = float("nan")
    mass = np.array([9, 1, 3, nan, 3, 2, 3, -1, 0.5, 8])
    assert oracle.evict_index(mass, 10, 5, 1, 1) == [0, 2, 4, 6, 9]    # three equal: all fit
    assert oracle.evict_index(mass, 10, 4, 1, 1) == [0, 2, 4, 9]       # two of them: the lower indices
    assert oracle.evict_index(mass, 10, 9, 1, 1) == [0, 1, 2, 4, 5, 6, 7, 8, 9]  # the NaN goes first
    assert oracle.evict_index(mass, 5, 5, 1, 1) == [0, 1, 2, 3, 4]
