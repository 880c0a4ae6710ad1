"""GPU parity of the key/value cache operators (softmax_ssa_fwd_b200.cache)
against their fp64 oracle (oracle/cache.py) on the same bf16 inputs.

Bounds, with H = 2^-8 (half a bf16 step, relative):
  append   one rounding to bf16 (H * |y|) after fp32 work: a sum of d squares, a
           reciprocal root and a rotation whose angle is off by at most 2^-24 of a
           half turn: 2^-18 of the size of the pair.
  tree     weights rounded to bf16 (H of the mean of |v| under the weights, A), the
           result rounded to bf16 (H * |out|); the fp32 sum of d products is
           off by at most d * 2^-23 * sum |q||k| * scale =: e whatever its order
           (2^-23, not 2^-24: the tensor cores may cut instead of round), which
           moves weights by 2 e relatively; exp2 and the sums: 2^-16.  lse: e + 2^-18.
  mass     e as above on each weight, 2^-22 of the exponent's terms
           (the products score * c, lse * c and exp2), a sum of at most 2^14
           terms in fp32 chains of at most 2^10: 2^-14.
  evict    exact.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oracle

pytestmark = pytest.mark.gpu

H = 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(scope="module")
def cache():
    from softmax_ssa_fwd_b200 import cache as mod
    return mod


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    from softmax_ssa_fwd_b200 import ssa
    assert ssa.ssa_device_status() == ssa.SSA_OK


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _near(got, want, tol, what=""):
    got = oracle.f64(got)
    assert got.shape == want.shape
    special = ~np.isfinite(want)
    assert np.array_equal(got[special], want[special], equal_nan=True), what
    over = np.abs(got[~special] - want[~special]) - np.broadcast_to(tol, want.shape)[~special]
    assert over.size == 0 or over.max() <= 0, (what, over.max())


# ------------------------------------------------------------------ append

APPEND = [
    # B, L, Hq, Hkv, d, rot, interleaved, axes, norm
    (1, 1, 1, 1, 64, 64, False, 1, "qk"),
    (1, 1, 32, 8, 128, 128, False, 1, "qk"),
    (8, 1, 32, 8, 128, 128, True, 1, ""),
    (3, 7, 6, 2, 128, 16, False, 1, "qk"),       # part of the head
    (2, 65, 7, 1, 64, 48, True, 3, "qk"),        # three axes, odd head count
    (1, 301, 5, 5, 128, 112, False, 4, "k"),     # only the keys are normalised
    (2, 33, 9, 3, 64, 0, False, 1, "q"),         # no rotation
    (1, 1500, 14, 2, 64, 32, False, 1, ""),
]


@pytest.mark.parametrize("B,L,Hq,Hkv,d,rot,pairs,axes,norm", APPEND)
def test_append(cache, B, L, Hq, Hkv, d, rot, pairs, axes, norm):
    cap = L + 5
    x = _rand(11 * B + L, B, L, Hq + 2 * Hkv, d)
    x[:, :, 0] *= 30  # sizes far from 1
    g = torch.Generator().manual_seed(L)
    wq = torch.randn(d, generator=g) if "q" in norm else None
    wk = torch.randn(d, generator=g) if "k" in norm else None
    pos = torch.randint(0, 3000000, (B, L, axes), generator=g, dtype=torch.int32)
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))
    axis = torch.arange(rot // 2, dtype=torch.int32) % axes
    start = _i32([b % 6 for b in range(B)])
    count = _i32([max(0, L - 2 * b) for b in range(B)])
    dev = [t.cuda() for t in x.split([Hq, Hkv, Hkv], 2)]  # (contiguous copies; strided below)
    base = x.cuda()
    q, k, v = base.split([Hq, Hkv, Hkv], 2)
    kc, vc = torch.full((B, cap, Hkv, d), 7.0).to(BF).cuda(), torch.full((B, cap, Hkv, d), 9.0).to(BF).cuda()
    out = torch.full((B, L, Hq, d), 5.0).to(BF).cuda()
    args = dict(inv_freq=freq, axis=axis, interleaved=pairs, factor=1.25, eps=1e-5, start=start.cuda(),
                count=count.cuda(), q_weight=None if wq is None else wq.cuda(),
                k_weight=None if wk is None else wk.cuda())
    if rot == 0:
        args["inv_freq"] = args["axis"] = None
    p = pos.cuda() if axes > 1 else pos[..., 0].contiguous().cuda()
    got = cache.append(q, k, v, kc, vc, p, out=out, **args)
    assert got is out
    want_q = np.full((B, L, Hq, d), 5.0)
    want_k, want_v = np.full((B, cap, Hkv, d), 7.0), np.full((B, cap, Hkv, d), 9.0)
    tol_q, tol_k = np.zeros_like(want_q), np.zeros_like(want_k)
    qn, kn, vn = (oracle.f64(t) for t in x.split([Hq, Hkv, Hkv], 2))
    for b in range(B):
        n, s = int(count[b]), int(start[b])
        f = freq.numpy()
        for src, w, dst, tol, rows in ((qn, wq, want_q, tol_q, slice(0, n)), (kn, wk, want_k, tol_k, slice(s, s + n))):
            y, size = oracle.rotate(src[b, :n], None if w is None else oracle.f64(w), pos[b, :n].numpy(), f,
                                    axis.numpy(), pairs, 1.25, 1e-5)
            dst[b, rows] = y
            tol[b, rows] = H * np.abs(y) + 2.0 ** -18 * size
        want_v[b, s:s + n] = vn[b, :n]
    _near(got, want_q, tol_q, "q")
    _near(kc, want_k, tol_k, "k")
    _near(vc, want_v, 0.0, "v")
    # contiguous inputs, written over q: the same bits
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    again = cache.append(*dev, kc2, vc2, p, out=dev[0], **args)
    for b in range(B):
        n, s = int(count[b]), int(start[b])
        assert torch.equal(again[b, :n], got[b, :n]) and torch.equal(kc2[b, s:s + n], kc[b, s:s + n])


def test_append_weights_need_four_byte_alignment_only(cache):
    B, L, Hq, Hkv, d = 1, 3, 2, 1, 64
    q, k, v = _rand(1, B, L, Hq, d).cuda(), _rand(2, B, L, Hkv, d).cuda(), _rand(3, B, L, Hkv, d).cuda()
    w = torch.randn(2 * d + 3, generator=torch.Generator().manual_seed(1)).cuda()
    kc = torch.zeros(2, B, L, Hkv, d, dtype=BF, device="cuda")
    one = cache.append(q, k, v, kc[0], kc[1], q_weight=w[1:1 + d], k_weight=w[d + 3:])
    also = cache.append(q, k, v, kc[1].clone(), kc[1], q_weight=w[1:1 + d].clone(), k_weight=w[d + 3:].clone())
    assert torch.equal(one, also)


def test_append_far_positions_and_rows_outside_the_cache(cache):
    # the same angle at far positions: 2^30 turns of a frequency that divides the circle differ from none
    L, d = 5, 64
    q, k, v = (_rand(i, 1, L, 2, d).cuda() for i in range(3))
    kc, vc = torch.zeros(1, 4, 2, d, dtype=BF, device="cuda"), torch.zeros(1, 4, 2, d, dtype=BF, device="cuda")
    freq = torch.full((d // 2,), 2 * np.pi / 1024, dtype=torch.float64)
    near = torch.arange(L, dtype=torch.int32)[None]
    a = cache.append(q, k, v, kc, vc, near.cuda(), inv_freq=freq, start=_i32([-2]).cuda())
    # rows -2, -1 and none past the end: tokens 2.. land at 0..
    y, size = oracle.rotate(oracle.f64(k)[0], None, near[0, :, None].numpy(), freq.numpy(), [0] * 32, False, 1.0, 0)
    _near(kc[0, :3], y[2:], H * np.abs(y[2:]) + 2.0 ** -18 * size[2:])
    assert torch.equal(vc[0, :3], v[0, 2:]) and not vc[0, 3].any()
    b = cache.append(q, k, v, kc, vc, (near + 2 ** 30).cuda(), inv_freq=freq, start=_i32([2]).cuda())
    # 2^20 whole turns; the double nearest 2 pi / 1024 is off by at most 2^-61: 2^-31 radians at 2^30
    _near(b, oracle.f64(a), 2 * H * np.abs(oracle.f64(a)) + 2.0 ** -17 * 5)
    assert torch.equal(vc[0, 2:], v[0, :2])


# ------------------------------------------------------------------ decode_tree

def _mask(kind, B, T, seed):
    r = np.random.RandomState(seed)
    bits = np.zeros((B, T, 32 * -(-T // 32)), bool)
    for b in range(B):
        for t in range(T):
            if kind == "chain":
                bits[b, t, :t + 1] = True
            elif kind == "tree":
                if t:
                    bits[b, t] = bits[b, r.randint(0, t)]
                bits[b, t, t] = True
            elif kind == "random":
                bits[b, t] = r.rand(bits.shape[2]) < 0.5  # bits past T are set as well
    return torch.from_numpy(np.packbits(bits, axis=-1, bitorder="little").view(np.int32))


def _tree(cache, q, k, v, lens, mask, scale=None, **kw):
    d = q.shape[3]
    scale = d ** -0.5 if scale is None else scale
    o, lse = cache.decode_tree(q.cuda(), k.cuda(), v.cuda(), lens.cuda(), mask.cuda(), scale=scale, **kw)
    return o, lse


def _tree_check(cache, q, k, v, lens, mask, scale=None, **kw):
    o, lse = _tree(cache, q, k, v, lens, mask, scale, **kw)
    d = q.shape[3]
    scale = d ** -0.5 if scale is None else scale
    with np.errstate(invalid="ignore", over="ignore"):
        wo, wl, absv, dots = oracle.decode_tree(q, k, v, lens, mask, scale)
    e = d * 2.0 ** -23 * scale * dots.max()
    fin = np.isfinite(absv)
    _near(o, wo, H * np.abs(np.where(fin, wo, 0)) + (H + 2 * e + 2.0 ** -16) * np.where(fin, absv, 0), "out")
    _near(lse, wl, e + 2.0 ** -18 * (1 + np.abs(np.where(np.isfinite(wl), wl, 0))), "lse")
    return o, lse


TREE = [
    # B, T, Hq, Hkv, d, lens, cap, kind
    (1, 1, 1, 1, 64, [0], 1, "chain"),                     # one key: the draft itself
    (4, 1, 32, 8, 128, [37, 600, 0, 127], 700, "chain"),
    (2, 1, 8, 1, 64, [1, 5000], 5001, "chain"),            # many blocks for one key head
    (3, 16, 8, 2, 128, [128, 1000, 112], 1024, "tree"),
    (2, 5, 7, 1, 64, [123, 124], 130, "chain"),            # G = 7; the draft crosses a tile's end
    (2, 33, 4, 4, 128, [200, 0], 256, "tree"),             # more than a mask word, G = 1
    (1, 61, 8, 2, 128, [700], 800, "tree"),                # two row tiles
    (2, 100, 8, 1, 64, [900, 30], 1000, "random"),         # several row groups
    (1, 128, 2, 2, 128, [1], 200, "random"),
    (1, 3, 128, 1, 64, [300], 310, "chain"),               # G = 128: a token a row tile
    (3, 9, 6, 2, 128, [50, 60, 500], 505, "none"),         # a row sees the cache only
    (40, 2, 4, 2, 64, [(17 * b) % 300 for b in range(40)], 302, "random"),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,d,lens,cap,kind", TREE)
def test_decode_tree(cache, B, T, Hq, Hkv, d, lens, cap, kind):
    q, k, v = _rand(1, B, T, Hq, d), _rand(2, B, cap, Hkv, d), _rand(3, B, cap, Hkv, d)
    lens, mask = _i32(lens), _mask(kind, B, T, T)
    first = _tree_check(cache, q, k, v, lens, mask)
    again = _tree(cache, q, k, v, lens, mask)
    assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("T", [4, 70])
@pytest.mark.parametrize("growing", [False, True])
def test_decode_tree_rescales(cache, growing, T):
    # scores that grow (or fall) along the keys, by more than a hundred in log2 units
    B, Hq, Hkv, d, n = 1, 4, 2, 64, 1500
    q, k, v = _rand(4, B, T, Hq, d), _rand(5, B, n + T, Hkv, d), _rand(6, B, n + T, Hkv, d)
    u = torch.zeros(d)
    u[0] = 1
    ramp = torch.linspace(-8, 8, n + T)[None, :, None, None] * (1 if growing else -1)
    q, k = (q + 20 * u).to(BF), (k + ramp * u).to(BF)
    _tree_check(cache, q, k, v, _i32([n]), _mask("chain", B, T, 0), scale=0.25)


def test_decode_tree_empty_rows(cache):
    B, T, Hq, Hkv, d, cap = 3, 4, 4, 2, 128, 300
    q, k, v = _rand(1, B, T, Hq, d), _rand(2, B, cap, Hkv, d), _rand(3, B, cap, Hkv, d)
    mask = _mask("chain", B, T, 0)
    mask[:, 1] = 0
    o, lse = _tree_check(cache, q, k, v, _i32([0, 5, 0]), mask)
    assert not o[0, 1].any() and torch.isinf(lse[0, :, 1]).all() and torch.isfinite(lse[1]).all()


def test_decode_tree_lengths_are_clamped(cache):
    # a negative length counts as 0, one past cap as cap (no draft row exists then)
    B, T, Hq, Hkv, d, cap = 4, 3, 4, 2, 64, 200
    q, k, v = _rand(1, B, T, Hq, d), _rand(2, B, cap, Hkv, d), _rand(3, B, cap, Hkv, d)
    _tree_check(cache, q, k, v, _i32([-7, 1000, 2 ** 31 - 1, 199]), _mask("chain", B, T, 0))


@pytest.mark.parametrize("d,T", [(64, 6), (128, 6), (128, 90)])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_decode_tree_hidden_values(cache, junk, d, T):
    """Rows past the draft and draft keys that a row does not see hold anything; a row that sees one gets it."""
    B, Hq, Hkv, cap = 2, 8, 2, 400
    lens = [120, 129]
    q, k, v = _rand(1, B, T, Hq, d), _rand(2, B, cap, Hkv, d), _rand(3, B, cap, Hkv, d)
    mask = _mask("chain", B, T, 0)
    clean = _tree(cache, q, k, v, _i32(lens), mask)
    k2, v2 = k.clone(), v.clone()
    for b in range(B):
        k2[b, lens[b] + T:], v2[b, lens[b] + T:] = junk, junk
        v2[b, lens[b] + T - 1] = junk          # the last draft key: seen by the last row only
        k2[b, lens[b] + T - 2, 0] = junk       # the last two rows
    o, lse = _tree(cache, q, k2, v2, _i32(lens), mask)
    assert torch.equal(o[:, :T - 2], clean[0][:, :T - 2]) and torch.equal(lse[..., :T - 2], clean[1][..., :T - 2])
    if not np.isfinite(junk):
        v3 = v.clone()
        for b in range(B):
            v3[b, lens[b] + T - 1] = junk
            v3[b, lens[b] + T - 1, :, d // 2:] = 1.5
        _tree_check(cache, q, k, v3, _i32(lens), mask)


def test_decode_tree_equals_decode(cache):
    """T = 1 over equal lengths is the dense decode step."""
    from softmax_ssa_fwd_b200 import ssa
    B, Hq, Hkv, d, L = 3, 16, 4, 128, 1111
    q, k, v = _rand(1, B, 1, Hq, d).cuda(), _rand(2, B, L, Hkv, d).cuda(), _rand(3, B, L, Hkv, d).cuda()
    o1, l1, _ = ssa.decode(q, k, v, lam=0.0, num_splits=4)
    o2, l2 = cache.decode_tree(q, k, v, _i32([L - 1] * B).cuda(), _i32([[[1]]] * B).cuda())
    assert (o1.float() - o2.float()).abs().max() <= 4 * H  # both within 2 H of |out| + A, both below 1
    assert (l1 - l2).abs().max() <= 1e-4


# ------------------------------------------------------------------ attn_mass

MASS = [
    # B, Lq, Hq, Hkv, d, lens, cap, causal, window, decay
    (1, 1, 1, 1, 64, [1], 1, True, 0, None),
    (3, 1, 8, 2, 128, [300, 5, 129], 301, True, 0, 1.0),
    (2, 4, 14, 2, 64, [500, 4], 520, True, 0, 0.5),
    (1, 64, 4, 1, 128, [700], 700, True, 0, None),         # 256 rows: the most of the streaming kernel
    (1, 65, 4, 1, 128, [700], 701, True, 0, 0.9),          # 260: the other one
    (2, 300, 8, 2, 64, [300, 411], 420, True, 0, None),
    (2, 300, 8, 2, 128, [300, 411], 420, False, 0, 1.0),
    (1, 257, 7, 1, 128, [257], 257, True, 0, None),        # G = 7
    (2, 500, 4, 2, 128, [500, 520], 600, True, 16, None),  # the last rows only
    (1, 3, 128, 1, 64, [200], 200, True, 0, None),         # G = 128
    (2, 20, 4, 4, 64, [0, 30], 300, True, 0, 1.0),         # nothing cached
    (1, 20, 2, 2, 64, [12], 40, True, 0, None),            # rows before the first key: left-padded
    (1, 300, 4, 2, 64, [100], 150, True, 0, None),         # the same with many rows
    (30, 3, 2, 1, 64, [(37 * b) % 500 for b in range(30)], 500, True, 0, 0.5),
]


def _lse(q, k, lens, causal, scale):
    qn, kn = oracle.f64(q), oracle.f64(k)
    B, Lq, Hq, d = qn.shape
    out = np.full((B, Hq, Lq), -np.inf)
    for b in range(B):
        n = int(lens[b])
        for h in range(Hq):
            x = scale * qn[b, :, h] @ kn[b, :n, h // (Hq // kn.shape[2])].T
            for i in range(Lq):
                m = min(n, i + n - Lq + 1) if causal else n
                if m > 0:
                    out[b, h, i] = np.logaddexp.reduce(x[i, :m])
    return torch.from_numpy(out).float()


@pytest.mark.parametrize("B,Lq,Hq,Hkv,d,lens,cap,causal,window,decay", MASS)
def test_attn_mass(cache, B, Lq, Hq, Hkv, d, lens, cap, causal, window, decay):
    q, k = _rand(1, B, Lq, Hq, d), _rand(2, B, cap, Hkv, d)
    lens, scale = _i32(lens), d ** -0.5
    lse = _lse(q, k, lens, causal, scale)
    mass = None if decay is None else torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(3))
    for b in range(B):  # past the length: anything
        k[b, int(lens[b]):] = float("nan")
        if mass is not None:
            mass[b, :, int(lens[b]):] = float("inf")
    kw = dict(lens=lens.cuda(), causal=causal, window=window, decay=1.0 if decay is None else decay)
    got = cache.attn_mass(q.cuda(), k.cuda(), lse.cuda(), mass=None if mass is None else mass.cuda(), **kw)
    want, dots, args = oracle.attn_mass(q, torch.nan_to_num(k.float()), lse, lens, causal, scale, window, mass, decay)
    _near(got, want, d * 2.0 ** -23 * dots + 2.0 ** -22 * args + 2.0 ** -14 * want, "mass")
    for b in range(B):
        assert not got[b, :, max(0, int(lens[b])):].any()
    if mass is not None:  # in place: the same bits
        m = mass.cuda()
        assert cache.attn_mass(q.cuda(), k.cuda(), lse.cuda(), mass=m, out=m, **kw) is m
        assert torch.equal(m, got)
    elif window == 0 and causal and int(lens.min()) >= Lq:  # every row's weights sum to 1
        total = got.sum((1, 2)).cpu()
        assert (total - Hq * Lq).abs().max() <= 1e-3 * Hq * Lq


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
@pytest.mark.parametrize("Lq", [3, 64, 200])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_mass_rows_without_keys_may_hold_anything(cache, causal, Lq, junk):
    B, Hq, Hkv, d, n = 1, 4, 1, 64, 333
    q, k, lens = _rand(1, B, Lq, Hq, d), _rand(2, B, n, Hkv, d), _i32([n])
    lse = _lse(q, k, lens, causal, 0.125)
    lse[:, 1, Lq // 2] = lse[:, :, 0] = -np.inf
    want, dots, args = oracle.attn_mass(q, k, lse, lens, causal, 0.125, 0, None, 1.0)
    q[:, Lq // 2, 1] = q[:, 0] = junk
    got = cache.attn_mass(q.cuda(), k.cuda(), lse.cuda(), lens=lens.cuda(), causal=causal)
    _near(got, want, d * 2.0 ** -23 * dots + 2.0 ** -22 * args + 2.0 ** -14 * want, "mass")


def test_attn_mass_of_an_infinite_key(cache):
    """Its score with the one row is -inf: no weight (rows that are not there must not make it NaN)."""
    q, k = torch.full((1, 1, 1, 64), -1.0).to(BF).cuda(), _rand(2, 1, 200, 1, 64).cuda()
    k[0, 7, 0, 3] = float("inf")
    got = cache.attn_mass(q, k, torch.zeros(1, 1, 1, device="cuda"), causal=False)
    assert got[0, 0, 7] == 0 and torch.isfinite(got).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("Lq,G", [(3, 4), (4, 4), (64, 4), (200, 4), (300, 7)])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_mass_of_rows_whose_lse_is_not_a_number(cache, causal, Lq, G, value):
    """A row with such a lse reaches the keys that it sees (NaN: makes them NaN; +inf: adds 0) and no others."""
    d, lens = 64, _i32([333, Lq // 2])  # the second sequence's first rows lie before its first key
    q, k = _rand(1, 2, Lq, G, d), _rand(2, 2, 340, 1, d)
    lse = _lse(q, k, lens, causal, 0.125)
    clean = cache.attn_mass(q.cuda(), k.cuda(), lse.cuda(), lens=lens.cuda(), causal=causal).cpu()
    lse[0, 1, Lq // 2] = lse[1, :, 0] = lse[1, 0, Lq - 2] = -np.inf
    _, dots, args = oracle.attn_mass(q, k, lse, lens, causal, 0.125, 0, None, 1.0)  # (the others' rounding)
    lse[0, 1, Lq // 2] = lse[1, :, 0] = lse[1, 0, Lq - 2] = value
    with np.errstate(invalid="ignore"):
        want, _, _ = oracle.attn_mass(q, k, lse, lens, causal, 0.125, 0, None, 1.0)
    got = cache.attn_mass(q.cuda(), k.cuda(), lse.cuda(), lens=lens.cuda(), causal=causal).cpu()
    _near(got, want, d * 2.0 ** -23 * dots + 2.0 ** -22 * args + 2.0 ** -14 * want, "mass")
    if np.isnan(value):
        hit = torch.zeros(2, 1, 340, dtype=torch.bool)
        hit[0, :, :333 - Lq + Lq // 2 + 1 if causal else 333] = True
        hit[1, :, :Lq // 2 - 1 if causal else Lq // 2] = True
        assert torch.equal(torch.isnan(got), hit)
        assert torch.equal(got[~hit], clean[~hit])


def test_attn_mass_of_an_infinite_score_and_lse(cache):
    """exp(inf - inf) is NaN on that key; the others have no weight beside it."""
    q, k = torch.full((1, 1, 1, 64), 1.0).to(BF).cuda(), _rand(2, 1, 200, 1, 64).cuda()
    k[0, 7, 0, 3] = float("inf")
    got = cache.attn_mass(q, k, torch.full((1, 1, 1), float("inf"), device="cuda"), causal=False)[0, 0].cpu()
    assert torch.isnan(got[7]) and not got[:7].any() and not got[8:].any()


@pytest.mark.parametrize("G", [8, 100])
def test_attn_mass_of_a_cache_of_millions_of_keys(cache, G):
    """One row of zeros with lse 0 gives every key a weight of one for each query head (100 heads, 22 million keys:
    a key's distance times the heads does not fit 32 bits)."""
    n = 22000000
    q, k = torch.zeros(1, 1, G, 64, dtype=BF, device="cuda"), torch.zeros(1, n, 1, 64, dtype=BF, device="cuda")
    got = cache.attn_mass(q, k, torch.zeros(1, G, 1, device="cuda"), lens=_i32([n - 5]).cuda())
    assert (got[..., :-5] == G).all() and not got[..., -5:].any()


@pytest.mark.parametrize("L", [50, 200])  # 200 and 800 rows a key head: both kernels
def test_attn_mass_of_prompts_padded_on_the_right(cache, L):
    """As `append` leaves them with count[b] < L: every length start[b] + L, and a lse of -inf in the padding's rows."""
    Hq, d, counts, start = 4, 64, [L, L // 3, 1], [0, 5, 20]
    q, k = _rand(1, 3, L, Hq, d), _rand(2, 3, L + 30, 1, d)
    lse = torch.full((3, Hq, L), -np.inf)
    want, tol = np.zeros((3, 1, L + 30)), np.zeros((3, 1, L + 30))
    for b, (n, s) in enumerate(zip(counts, start)):
        one = q[b:b + 1, :n], k[b:b + 1], _i32([s + n])
        lse[b:b + 1, :, :n] = _lse(*one, True, 0.125)
        want[b:b + 1], dots, args = oracle.attn_mass(*one[:2], lse[b:b + 1, :, :n], one[2], True, 0.125, 0, None, 1.0)
        tol[b:b + 1] = d * 2.0 ** -23 * dots + 2.0 ** -22 * args + 2.0 ** -14 * want[b:b + 1]
        q[b, n:], k[b, s + n:] = float("nan"), float("nan")
    got = cache.attn_mass(q.cuda(), k.cuda(), lse.cuda(), lens=_i32([s + L for s in start]).cuda())
    _near(got, want, tol, "mass")


def test_attn_mass_counts_keys_that_the_attention_left_out(cache):
    """A chain's rows give the weights of decode_tree, a row of one sum 1; a tree's rows also count the branches that they
    do not see, as a causal row does."""
    B, T, Hq, Hkv, d, n = 1, 3, 2, 1, 64, 100
    q, k, v = _rand(1, B, T, Hq, d).cuda(), _rand(2, B, n + T, Hkv, d).cuda(), _rand(3, B, n + T, Hkv, d).cuda()
    lens = _i32([n]).cuda()
    for mask, least in ((_mask("chain", B, T, 0), 0.0), (_i32([[[1], [2], [4]]]), 1e-3)):  # three branches of one token
        _, lse = cache.decode_tree(q, k, v, lens, mask.cuda())
        over = cache.attn_mass(q, k, lse, lens=lens + T).double().sum().item() - Hq * T
        x = torch.einsum("ihd,jd->hij", q[0].double(), k[0, :, 0].double()) * d ** -0.5
        x = torch.exp(x - lse[0].double()[..., None]).tril(n).sum().item() - Hq * T
        assert abs(over - x) <= 1e-3 and (over >= least if least else abs(over) <= 1e-3)


# ------------------------------------------------------------------ evict

EVICT = [
    # B, Hkv, d, lens, cap, keep, sink, recent, cap_out
    (1, 1, 64, [1], 1, 1, 0, 0, 1),
    (3, 2, 64, [200, 450, 700], 700, 257, 4, 33, 300),
    (2, 4, 128, [0, 90], 100, 64, 0, 0, 64),
    (2, 1, 128, [5000, 2999], 5000, 1000, 0, 1000, 1000),     # only recent ones
    (1, 2, 64, [6000], 6000, 100, 100, 0, 110),               # only first ones
    (1, 1, 64, [50000], 50000, 20001, 3, 17, 20001),          # a slice past one block's shared memory / a cluster
    (1, 8, 128, [33000], 33333, 1, 0, 0, 1),
    (70, 2, 64, [(31 * b) % 300 for b in range(70)], 300, 100, 1, 2, 100),
    (38, 2, 64, [45000] * 38, 45000, 5, 1, 1, 5),             # one block a head, masses past its shared memory
]


@pytest.mark.parametrize("B,Hkv,d,lens,cap,keep,sink,recent,cap_out", EVICT)
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict(cache, B, Hkv, d, lens, cap, keep, sink, recent, cap_out, kind):
    if B * cap > 10 ** 6 and kind != "ties":
        pytest.skip("one kind is enough at this size")
    g = torch.Generator().manual_seed(cap)
    mass = torch.rand(B, Hkv, cap, generator=g)
    if kind == "ties":
        mass = (mass * 3).floor() / 7  # three values
    if kind == "odd":
        mass = torch.where(mass < 0.3, -mass, mass)
        for x, f in ((0.4, 0.0), (0.5, -0.0), (0.6, float("nan")), (0.62, float("inf")), (0.7, -float("inf")),
                     (0.72, 1e-40), (0.74, 2e-40)):
            mass = torch.where((mass > x - 0.01) & (mass < x), torch.full_like(mass, f), mass)
    j = torch.arange(cap, dtype=torch.int32)[None, :, None]
    tag = torch.stack([j + 0 * torch.zeros(B, cap, Hkv, dtype=torch.int32), j * 0 + torch.arange(B)[:, None, None].int()
                       + torch.zeros(B, cap, Hkv, dtype=torch.int32)], -1)  # every row of k, v names itself
    k = torch.zeros(B, cap, Hkv, d, dtype=BF)
    k.view(torch.int16)[..., :2] = tag.short()
    v = k.clone()
    v.view(torch.int16)[..., d - 1] = torch.arange(Hkv, dtype=torch.int16)
    k.view(torch.int16)[..., 2] = torch.arange(Hkv, dtype=torch.int16)
    ko, vo = (torch.full((B, cap_out, Hkv, d), 3.0, dtype=BF, device="cuda") for _ in range(2))
    got = cache.evict(k.cuda(), v.cuda(), mass.cuda(), _i32(lens).cuda(), keep=keep, sink=sink, recent=recent, k_out=ko,
                      v_out=vo)
    mn, index, mo = mass.numpy(), got.index.cpu(), got.mass.cpu()
    gk, gv = ko.cpu(), vo.cpu()
    assert got.lens.tolist() == [min(n, keep) for n in lens]
    for b in range(B):
        for h in range(Hkv):
            want = oracle.evict_index(mn[b, h], lens[b], keep, sink, recent)
            n = len(want)
            assert index[b, h].tolist() == want + [-1] * (keep - n), (b, h)
            assert torch.equal(mo[b, h, :n].view(torch.int32), mass[b, h, want].view(torch.int32))
            assert not mo[b, h, n:].any()
            assert torch.equal(gk[b, :n, h].view(torch.int16), k[b, want, h].view(torch.int16))
            assert torch.equal(gv[b, :n, h].view(torch.int16), v[b, want, h].view(torch.int16))
            assert (gk[b, n:, h] == 3).all() and (gv[b, n:, h] == 3).all()


# ------------------------------------------------------------------ together

def test_a_generation(cache):
    """Prompt, mass of its last rows, eviction, drafted tokens: against the oracle on what the cache holds."""
    from softmax_ssa_fwd_b200 import ssa
    B, L, Hq, Hkv, d, cap, T = 2, 700, 8, 2, 128, 720, 5
    x = _rand(5, B, L + T, Hq + 2 * Hkv, d).cuda()
    freq, factor = cache.rope_frequencies(d, 5e5, scaling="bands", factor=8.0)
    kc = torch.full((B, cap, Hkv, d), float("nan"), dtype=BF, device="cuda")
    vc = kc.clone()
    pos = torch.arange(L + T, dtype=torch.int32, device="cuda")[None].repeat(B, 1)
    split = lambda y: y.split([Hq, Hkv, Hkv], 2)  # noqa: E731
    q = cache.append(*split(x[:, :L]), kc, vc, pos[:, :L].contiguous(), inv_freq=freq, factor=factor)
    kp, vp = kc[:, :L].contiguous(), vc[:, :L].contiguous()
    out, lse, _ = ssa.attention(q, kp, vp, causal=True, mode=ssa.MODE_DENSE)
    lens = _i32([L] * B).cuda()
    mass = cache.attn_mass(q, kc, lse, lens=lens, window=32)
    total = mass.sum((1, 2))
    assert (total - 32 * Hq).abs().max() <= 0.02 * 32 * Hq  # lse of the attention: within 1e-3 of exact, bf16 inputs alike
    keep = 200
    ko = torch.full((B, keep + 40, Hkv, d), float("nan"), dtype=BF, device="cuda")
    small = cache.evict(kc, vc, mass, lens, keep=keep, sink=4, recent=32, k_out=ko, v_out=ko.clone())
    for b in range(B):
        for h in range(Hkv):
            want = oracle.evict_index(mass[b, h].cpu().numpy(), L, keep, 4, 32)
            assert small.index[b, h].tolist() == want
    # the draft: positions go on from the prompt's, rows from the small cache's length
    mask = _mask("tree", B, T, 3).cuda()
    qt = cache.append(*split(x[:, L:]), small.k, small.v, pos[:, L:].contiguous(), inv_freq=freq, factor=factor,
                      start=small.lens)
    o, lse = cache.decode_tree(qt, small.k, small.v, small.lens, mask)
    assert torch.isfinite(o).all()
    _tree_check(cache, qt, torch.nan_to_num(small.k), torch.nan_to_num(small.v), small.lens.cpu(), mask)
    # weight of the draft's last token, onto the kept masses
    more = cache.attn_mass(qt[:, -1:].contiguous(), small.k, lse[..., -1:].contiguous(), lens=small.lens + T,
                           mass=small.mass, decay=0.5)
    assert more.shape == small.mass.shape and torch.isfinite(more).all()


def test_offsets_past_32_bits(cache):
    """The second sequence of a cache of 2.9e9 elements gives what it gives on its own."""
    B, T, Hq, Hkv, d, cap = 2, 2, 32, 16, 128, 700000
    k, v = torch.zeros(B, cap, Hkv, d, dtype=BF, device="cuda"), torch.zeros(B, cap, Hkv, d, dtype=BF, device="cuda")
    x = _rand(1, B, T, Hq + 2 * Hkv, d).cuda()
    qkv = x.split([Hq, Hkv, Hkv], 2)
    k[1, -300:] = 2 * _rand(2, 300, Hkv, d).cuda()
    v[1, -300:] = _rand(3, 300, Hkv, d).cuda()
    lens = _i32([5, cap - T]).cuda()
    q = cache.append(*qkv, k, v, start=lens)
    assert torch.equal(k[1, -T:], qkv[1][1]) and torch.equal(v[1, -T:], qkv[2][1]) and torch.equal(k[0, 5:7], qkv[1][0])
    mask = _mask("chain", B, T, 0).cuda()
    o, lse = cache.decode_tree(q, k, v, lens, mask)
    o1, lse1 = cache.decode_tree(q[1:], k[1:], v[1:], lens[1:], mask[1:])
    # the same sums cut elsewhere: two roundings of the weights and the result, values below 5
    assert (o[1:].float() - o1.float()).abs().max() <= 4 * H * 5 and (lse[1:] - lse1).abs().max() <= 2.0 ** -14
    m = cache.attn_mass(q, k, lse, lens=lens + T)
    m1 = cache.attn_mass(q[1:], k[1:], lse[1:], lens=lens[1:] + T)
    assert torch.equal(m[1:], m1) and (m.sum((1, 2)) - Hq * T).abs().max() <= 0.01 * Hq * T
    small, one = (cache.evict(a, b, c, n, keep=64, sink=1, recent=2) for a, b, c, n in
                  ((k, v, m, lens + T), (k[1:], v[1:], m1, lens[1:] + T)))
    assert torch.equal(small.index[1:], one.index) and torch.equal(small.k[1:], one.k) and torch.equal(small.v[1:], one.v)
    assert one.index[0, :, -1].tolist() == [cap - 1] * Hkv
    assert torch.equal(one.k[0, -1], k[1, -1]) and torch.equal(one.v[0, -1], v[1, -1])


def test_as_many_sequences_as_allowed(cache):
    B, T, Hq, Hkv, d, cap = 1024, 1, 2, 1, 64, 260
    q, k, v = _rand(1, B, T, Hq, d), _rand(2, B, cap, Hkv, d), _rand(3, B, cap, Hkv, d)
    lens = _i32([(37 * b) % 260 for b in range(B)])
    o, lse = _tree_check(cache, q, k, v, lens, _mask("chain", B, T, 0))
    got = cache.attn_mass(q.cuda(), k.cuda(), lse, lens=lens.cuda() + 1).sum((1, 2))
    assert (got - Hq).abs().max() <= 1e-3


def test_replay_reads_the_lengths_of_the_moment(cache):
    B, T, Hq, Hkv, d, cap = 2, 3, 8, 2, 128, 900
    q, k, v = _rand(1, B, T, Hq, d).cuda(), _rand(2, B, cap, Hkv, d).cuda(), _rand(3, B, cap, Hkv, d).cuda()
    lens, mask = _i32([100, 800]).cuda(), _mask("chain", B, T, 0).cuda()
    mass = torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(3)).cuda()

    def step():
        o, lse = cache.decode_tree(q, k, v, lens, mask)
        m = cache.attn_mass(q, k, lse, lens=lens + T, mass=mass, decay=0.5)
        e = cache.evict(k, v, m, lens, keep=90, sink=2, recent=9)
        return [o, lse, m, e.index, e.lens, e.mass]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
    for now in ([100, 800], [897, 3], [0, 500]):
        lens.copy_(_i32(now))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for x, y in zip(got, step()):
            assert torch.equal(x, y), now


def test_two_streams_at_once(cache):
    """Calls in flight on two streams do not share scratch memory."""
    B, T, Hq, Hkv, d, cap = 4, 8, 8, 2, 128, 4000
    mask = _mask("chain", B, T, 0).cuda()
    lens = _i32([3990, 100, 2000, 0]).cuda()
    sets = [[_rand(s, B, T, Hq, d).cuda(), _rand(s + 1, B, cap, Hkv, d).cuda(), _rand(s + 2, B, cap, Hkv, d).cuda()]
            for s in (1, 5)]
    want = [cache.decode_tree(*s, lens, mask) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for n, st in enumerate(streams):
            got[n].append(cache.decode_tree(*sets[n], lens, mask, stream=st if _ % 2 else st.cuda_stream))
    torch.cuda.synchronize()
    for n in range(2):
        for o, lse in got[n]:
            assert torch.equal(o, want[n][0]) and torch.equal(lse, want[n][1])


def test_waits_that_run_out_are_reported(cache):
    """A limit of one nanosecond: blocks give up, the call returns, ssa_device_status says so, the next call is right."""
    from softmax_ssa_fwd_b200 import ssa
    B, T, Hq, Hkv, d, cap = 4, 8, 8, 2, 128, 4000
    q, k, v = _rand(1, B, T, Hq, d).cuda(), _rand(2, B, cap, Hkv, d).cuda(), _rand(3, B, cap, Hkv, d).cuda()
    lens, mask = _i32([3990, 100, 2000, 0]).cuda(), _mask("chain", B, T, 0).cuda()
    o, lse = cache.decode_tree(q, k, v, lens, mask)
    qm = _rand(4, B, 100, Hq, d).cuda()
    lm = torch.zeros(B, Hq, 100, device="cuda")
    m = cache.attn_mass(q, k, lse, lens=lens), cache.attn_mass(qm, k, lm, lens=lens)
    torch.cuda.synchronize()
    for call in (lambda: cache.decode_tree(q, k, v, lens, mask), lambda: cache.attn_mass(q, k, lse, lens=lens),
                 lambda: cache.attn_mass(qm, k, lm, lens=lens)):
        ssa.ssa_set_wait_timeout_ns(1)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            ssa.ssa_set_wait_timeout_ns(0)
        assert ssa.ssa_device_status() == ssa.SSA_ERR_TIMEOUT
        assert ssa.ssa_device_status() == ssa.SSA_OK
    o2, lse2 = cache.decode_tree(q, k, v, lens, mask)
    m2 = cache.attn_mass(q, k, lse, lens=lens), cache.attn_mass(qm, k, lm, lens=lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(m[0], m2[0]) and torch.equal(m[1], m2[1])


@pytest.mark.parametrize("ns", [2 ** 63, 2 ** 64 - 1])
def test_a_limit_longer_than_the_clock_counts(cache, ns):
    """Limits that stand for none do not run out at once."""
    from softmax_ssa_fwd_b200 import ssa
    B, T, Hq, Hkv, d, cap = 2, 8, 8, 2, 128, 2000
    q, k, v = _rand(1, B, T, Hq, d).cuda(), _rand(2, B, cap, Hkv, d).cuda(), _rand(3, B, cap, Hkv, d).cuda()
    lens, mask = _i32([1990, 100]).cuda(), _mask("chain", B, T, 0).cuda()
    qm, lm = _rand(4, B, 100, Hq, d).cuda(), torch.zeros(B, Hq, 100, device="cuda")

    def call():
        o, lse = cache.decode_tree(q, k, v, lens, mask)
        return o, lse, cache.attn_mass(q, k, lse, lens=lens), cache.attn_mass(qm, k, lm, lens=lens)

    want = call()
    ssa.ssa_set_wait_timeout_ns(ns)
    try:
        got = call()
        torch.cuda.synchronize()
    finally:
        ssa.ssa_set_wait_timeout_ns(0)
    assert ssa.ssa_device_status() == ssa.SSA_OK
    assert all(torch.equal(x, y) for x, y in zip(got, want))
