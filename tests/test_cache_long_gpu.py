"""GPU tests of the cache operators where a block walks several tiles of a segment
and several segments (many more tiles than SMs), against a plain implementation
in 64 bits on the GPU, and of how the operators are called: captured, from
other threads, with a workspace of the caller's.

Bounds as in test_cache_gpu.py (H = 2^-8, A the mean of |v| under the weights,
e = d * 2^-23 * scale * max |q||k|), with the terms that grow with the length:
at most 2^6 additions of 16 products each to an accumulator of a block, which may cut
(2^-23 each: 2^-17), at most 2^4 rescalings (2^-22 each: 2^-18) and the merge
of the parts (2^-20): 2^-15 A in all for the result, 2^-16 for the log-sum-exp.
"""
import threading

import numpy as np
import pytest
import torch

from test_cache_gpu import BF, H, _i32, _mask, _near, _no_wait_gave_up, _rand, cache  # noqa: F401

pytestmark = pytest.mark.gpu


def _tree64(q, k, v, lens, mask, scale):
    """(out, lse, mean of |v| under the weights, largest sum of |q||k|) in 64 bits, one key head at a time."""
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    bits = np.unpackbits(np.ascontiguousarray(mask.cpu().numpy()).view(np.uint8), axis=-1, bitorder="little")
    bits = torch.from_numpy(bits[..., :T].astype(bool)).cuda()
    f64 = dict(dtype=torch.float64, device="cuda")
    out, absv = torch.zeros(B, T, Hq, d, **f64), torch.zeros(B, T, Hq, d, **f64)
    lse, dots = torch.zeros(B, Hq, T, **f64), torch.zeros(B, Hq, T, **f64)
    for b in range(B):
        n = int(lens[b])
        sees = torch.ones(T, n + T, dtype=torch.bool, device="cuda")
        sees[:, n:] = bits[b]
        for h in range(Hkv):
            hq = slice(h * G, (h + 1) * G)
            qq, kk, vv = q[b, :, hq].double(), k[b, :n + T, h].double(), v[b, :n + T, h].double()
            x = (torch.einsum("tgd,jd->gtj", qq, kk) * scale).masked_fill(~sees, -np.inf)
            lse[b, hq] = torch.logsumexp(x, -1)
            w = torch.softmax(x, -1)
            out[b, :, hq], absv[b, :, hq] = (torch.einsum("gtj,jd->tgd", w, u) for u in (vv, vv.abs()))
            dots[b, hq] = (qq.abs() @ kk.abs().T).amax(-1).T
    return out, lse, absv, dots


def _check(got, q, k, v, lens, mask, scale, sums=2.0 ** -15, lse_sums=2.0 ** -16):
    out, lse, absv, dots = (t.cpu().numpy() for t in _tree64(q, k, v, lens, mask, scale))
    e = q.shape[3] * 2.0 ** -23 * scale * dots  # [B, Hq, T]
    e_row = e.transpose(0, 2, 1)[..., None]
    _near(got[0], out, H * np.abs(out) + (H + 2 * e_row + sums) * absv, "out")
    _near(got[1], lse, e + lse_sums + 2.0 ** -18 * np.abs(lse), "lse")


LENS = [128 * 70 + 100, 128 * 23 + 100, 128 * 60 + 100, 128 * 40 + 100]  # the draft shares its tile with 100 keys
HKV = 8
LONG = [  # T, query heads a key head, d: rows a key head and the kernel form they take
    (1, 8, 128), (2, 4, 64),     # 8: few rows, 16 columns
    (4, 8, 64), (2, 16, 128),    # 32: few rows, 32 columns
    (7, 6, 128), (5, 8, 64),     # 42 and 40: many rows, one row tile, not full
    (16, 4, 64), (18, 7, 128),   # 64, 126
    (61, 4, 128), (36, 7, 64),   # 244, 252: two row tiles, not full
    (40, 7, 64),                 # 280: two row groups
]


def _long(T, G, d, ramp):
    """Scores that rise along the keys for every second row and fall for the others, by `ramp` * 2 before scaling."""
    B, cap = len(LENS), max(LENS) + T + 3
    tiles = HKV * sum(-(-(n + T) // 128) for n in LENS)
    # so that blocks walk several tiles of a segment, and two segments
    assert tiles >= 4 * torch.cuda.get_device_properties(0).multi_processor_count
    q, k, v = (_rand(T + i, *s, d).cuda() for i, s in enumerate(((B, T, HKV * G), (B, cap, HKV), (B, cap, HKV))))
    sign = torch.tensor([-1.0, 1.0]).repeat(T * HKV * G + 1)[:T * HKV * G].view(T, HKV * G).cuda()
    q[..., 0] += (20 * sign).to(BF)
    k[..., 0] += torch.linspace(-ramp / 20, ramp / 20, cap, device="cuda")[None, :, None].to(BF)
    return q, k, v, _i32(LENS).cuda()


@pytest.mark.parametrize("T,G,d", LONG)
@pytest.mark.parametrize("ramp", [0, 160])
def test_decode_tree_of_many_tiles(cache, T, G, d, ramp):  # noqa: F811
    """Ramp 160, scale 1/4: scores move by 80 along the keys, so rows rescale again and again, each at its own tiles."""
    q, k, v, lens = _long(T, G, d, ramp)
    mask = _mask("tree", len(LENS), T, T).cuda()
    scale = 0.25 if ramp else d ** -0.5
    got = cache.decode_tree(q, k, v, lens, mask, scale=scale)
    _check(got, q, k, v, lens, mask, scale)
    again = cache.decode_tree(q, k, v, lens, mask, scale=scale)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("T,G,d,before", [(7, 6, 128, 16), (5, 8, 64, 16), (18, 7, 128, 16), (36, 7, 64, 32)])
def test_decode_tree_does_not_depend_on_what_ran_before(cache, T, G, d, before):  # noqa: F811
    """The same bits after a call that leaves zeros in shared memory and after one that leaves large queries there."""
    q, k, v, lens = _long(T, G, d, 0)
    mask = _mask("chain", len(LENS), T, 0).cuda()
    fill, fill_mask = 100 * _rand(9, len(LENS), before, HKV * 8, d).cuda(), _mask("chain", len(LENS), before, 0).cuda()
    got = []
    for x in (torch.zeros_like(fill), fill):
        cache.decode_tree(x, k, v, lens, fill_mask)
        got.append(cache.decode_tree(q, k, v, lens, mask))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("T,G,d", [t for t in LONG if t[0] > 1])
@pytest.mark.parametrize("junk", ["aligned", float("nan"), float("inf"), 3e38])
def test_decode_tree_hidden_keys_of_later_tiles(cache, T, G, d, junk):  # noqa: F811
    """The last draft key, seen by the last row only, and what lies past the draft leave the others' bits alone.
    "aligned": a score of about 45 for a row that sees the key, far ahead of every other key's."""
    q, k, v, lens = _long(T, G, d, 20)  # rising: later tiles often bring a new, little larger, maximum
    mask = _mask("chain", len(LENS), T, 0).cuda()
    clean = cache.decode_tree(q, k, v, lens, mask)
    for b, n in enumerate(LENS):
        at = n + T - 1
        if junk == "aligned":
            x = q[b, T - 1].view(HKV, G, d)[:, 0].float()
            k[b, at] = (x * 45 * d ** 0.5 / x.square().sum(-1, keepdim=True)).to(BF)
            v[b, at] *= 100
        else:
            k[b, at] = v[b, at] = junk
            k[b, at + 1:] = v[b, at + 1:] = junk
    got = cache.decode_tree(q, k, v, lens, mask)
    assert torch.equal(got[0][:, :T - 1], clean[0][:, :T - 1])
    assert torch.equal(got[1][..., :T - 1], clean[1][..., :T - 1])
    if junk == "aligned":
        _check(got, q, k, v, lens, mask, d ** -0.5)


# ------------------------------------------------------------------ offsets past 32 bits

@pytest.mark.parametrize("T,Hq", [(2, 32), (16, 64)])  # 4 rows a key head: few rows; 64: many
def test_decode_tree_past_32_bits_against_64_bits(cache, T, Hq):  # noqa: F811
    """The second sequence of a cache of 2.9e9 elements, whose last 300 keys hold much of the weight."""
    B, Hkv, d, cap = 2, 16, 128, 700000
    k, v = torch.zeros(B, cap, Hkv, d, dtype=BF, device="cuda"), torch.zeros(B, cap, Hkv, d, dtype=BF, device="cuda")
    q = _rand(1, B, T, Hq, d).cuda()
    k[1, -300:] = 5 * _rand(2, 300, Hkv, d).cuda()
    v[1, -300:] = _rand(3, 300, Hkv, d).cuda()
    lens, mask = _i32([5, cap - T]).cuda(), _mask("chain", B, T, 0).cuda()
    got = cache.decode_tree(q, k, v, lens, mask)
    # 592 tiles a block, 296 a group: 2368 additions to an accumulator, 2^-23 each; 296 + 2^5 to a row's sum, 2^-24 each
    _check([got[0][1:], got[1][1:]], q[1:], k[1:], v[1:], lens[1:], mask[1:], d ** -0.5, 2.0 ** -11, 2.0 ** -15)


# ------------------------------------------------------------------ how they are called

def test_append_replays_with_the_tensors_of_the_moment(cache):  # noqa: F811
    """A captured append keeps its table of frequencies (by value) and reads positions, starts and counts anew."""
    B, L, Hq, Hkv, d, cap = 2, 5, 8, 2, 128, 64
    x = _rand(1, B, L, Hq + 2 * Hkv, d).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], 2)
    freq, factor = cache.rope_frequencies(d, 5e5, scaling="bands", factor=8.0)
    kept = freq.clone()
    pos, start, count = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, L), (B,), (B,)))
    w = torch.randn(d, generator=torch.Generator().manual_seed(1)).cuda()

    def call(f, kc, vc, out):
        return cache.append(q, k, v, kc, vc, pos, inv_freq=f, factor=factor, q_weight=w, k_weight=w, start=start,
                            count=count, out=out)

    held, want = ([torch.zeros(B, n, h, d, dtype=BF, device="cuda") for n, h in ((cap, Hkv), (cap, Hkv), (L, Hq))]
                  for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    call(freq, *want)
    with torch.cuda.graph(graph):
        call(freq, *held)
    freq.zero_()
    for p0, s, c in ((7, [0, 9], [5, 5]), (100000, [60, 3], [5, 2]), (0, [-2, 20], [0, 9])):
        pos.copy_(torch.arange(L, dtype=torch.int32)[None] + p0)
        start.copy_(_i32(s))
        count.copy_(_i32(c))
        x.copy_(_rand(p0 + 2, B, L, Hq + 2 * Hkv, d))
        for t in held + want:
            t.zero_()
        graph.replay()
        call(kept, *want)
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        assert want[0].any()


@pytest.mark.parametrize("T", [3, 20])
def test_decode_tree_in_a_workspace_of_the_caller(cache, T):  # noqa: F811
    from softmax_ssa_fwd_b200 import ssa
    B, Hq, Hkv, d, cap = 2, 8, 2, 128, 900
    q, k, v = _rand(1, B, T, Hq, d).cuda(), _rand(2, B, cap, Hkv, d).cuda(), _rand(3, B, cap, Hkv, d).cuda()
    lens, mask = _i32([100, 800]).cuda(), _mask("chain", B, T, 0).cuda()
    want = cache.decode_tree(q, k, v, lens, mask)
    n = cache.ssa_decode_tree_workspace_bytes(B, T, Hq, Hkv, cap, d)
    room = torch.full((n + 256,), 0x7f, dtype=torch.uint8, device="cuda")  # junk before, a guard behind
    for _ in range(2):
        got = cache.decode_tree(q, k, v, lens, mask, workspace=room[:n])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (room[n:] == 0x7f).all()
    for bad in (room[:n - 1], room[8:n + 8], room[:n].cpu(), room[:2 * (n // 2)].view(-1, 2)[:, 0]):
        with pytest.raises(ssa.SSAError) as e:
            cache.decode_tree(q, k, v, lens, mask, workspace=bad)
        assert e.value.status == ssa.SSA_ERR_INVALID_ARG


def test_calls_from_other_threads(cache):  # noqa: F811
    """Two threads on streams of their own, at once: what one thread gets alone."""
    B, T, Hq, Hkv, d, cap = 2, 4, 8, 2, 64, 2000
    mask, lens = _mask("chain", B, T, 0).cuda(), _i32([1990, 700]).cuda()
    freq, _ = cache.rope_frequencies(d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)

    def steps(seed):
        k, v = _rand(seed, B, cap, Hkv, d).cuda(), _rand(seed + 1, B, cap, Hkv, d).cuda()
        q, kn, vn = _rand(seed + 2, B, T, Hq + 2 * Hkv, d).cuda().split([Hq, Hkv, Hkv], 2)
        q = cache.append(q, kn, vn, k, v, pos, inv_freq=freq, start=lens)
        out, lse = cache.decode_tree(q, k, v, lens, mask)
        mass = cache.attn_mass(q, k, lse, lens=lens + T)
        return [out, lse, mass, *cache.evict(k, v, mass, lens, keep=600, sink=2, recent=9)]

    want = [steps(s) for s in (1, 11)]
    torch.cuda.synchronize()
    got, failed = [None, None], []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[n] = steps((1, 11)[n])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_readme_generation(cache):  # noqa: F811
    """The example as printed: the drafted tokens are in the small cache, and the rows see them."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    prompt, step = next(b for b in blocks if "cache.evict" in b).split("# then, per step")
    B, L, Hq, Hkv, d, T = 2, 4200, 4, 2, 128, 6
    zeros = lambda: torch.zeros(B, L, Hkv, d, dtype=BF, device="cuda")  # noqa: E731
    pos = torch.arange(L + T, dtype=torch.int32, device="cuda").repeat(B, 1)
    x = _rand(5, B, L + T, Hq + 2 * Hkv, d).cuda()
    env = dict(zip("qkv", x[:, :L].split([Hq, Hkv, Hkv], 2)), k_cache=zeros(), v_cache=zeros(), lens=_i32([L] * B).cuda(),
               positions=pos[:, :L].contiguous(), wq=torch.ones(d, device="cuda"), wk=torch.ones(d, device="cuda"))
    exec(prompt, env)
    lens = env["small"].lens.clone()
    assert lens.tolist() == [4096] * B
    env.update(zip("qkv", x[:, L:].split([Hq, Hkv, Hkv], 2)), positions=pos[:, L:].contiguous(),
               tree_mask=_mask("tree", B, T, 3).cuda(), accepted=_i32([3, 1]).cuda())
    exec("# then, per step" + step, env)
    small = env["small"]
    assert small.lens.tolist() == [4099, 4097] and torch.equal(small.v[:, 4096:4096 + T], x[:, L:, Hq + Hkv:])
    _check([env["out"], env["lse"]], env["q"], small.k, small.v, lens, env["tree_mask"], d ** -0.5)
