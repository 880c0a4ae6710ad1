"""The operators around the key/value cache, as they are called, with their plain forms.

append       per-head norm of queries and keys, position rotation, and the write of keys and values into the cache
decode_tree  attention of drafted tokens (a tree, a chain or one token) over caches of different lengths
attn_mass    attention weight that each cached key received, accumulated
evict        compaction of a cache to its heaviest keys

``own`` False: elementary torch operations in 32 bits (64 for the angles).  True: softmax_ssa_fwd_b200.cache.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one new token of each of 8 sequences around position 32k, Qwen3-8B heads: a decode step's latency
        dict(name="append token b8", op="append", B=8, L=1, Hq=32, Hkv=8, d=128, rot=128, layout="half", norm=True,
             axes=1, base=1e6, stretch=1.0, factor=1.0, far=32700, cap=4096, ragged=False),
        # a whole 8k prompt of the Llama-3.1-8B shape, no norm, stretched frequencies (long-context scaling)
        dict(name="append prompt 8k", op="append", B=1, L=8192, Hq=32, Hkv=8, d=128, rot=128, layout="half", norm=False,
             axes=1, base=5e5, stretch=8.0, factor=1.0, far=0, cap=8192, ragged=False),
        # a padded batch of chunks, d = 64, interleaved pairs over half of the head, positions past a million
        dict(name="append ragged chunk", op="append", B=5, L=777, Hq=14, Hkv=2, d=64, rot=32, layout="pairs", norm=True,
             axes=1, base=1e4, stretch=32.0, factor=1.2, far=1000003, cap=2048, ragged=True),
        # the video shape: 21 x 45 x 80 tokens, 40 heads, three axes, interleaved pairs; the largest
        dict(name="append video 75600", op="append", B=1, L=75600, Hq=40, Hkv=40, d=128, rot=128, layout="pairs",
             norm=True, axes=3, base=1e4, stretch=1.0, factor=1.0, far=0, cap=75600, ragged=False),
        # one token of each of 4 short chats: latency
        dict(name="tree token short", op="tree", B=4, T=1, Hq=32, Hkv=8, d=128, lo=37, hi=600),
        # the decode workload's shape with a draft of 16 and caches between a third and all of 32k
        dict(name="tree t16 32k", op="tree", B=8, T=16, Hq=32, Hkv=8, d=128, lo=11000, hi=32768),
        # a wide tree (244 query rows a key head) over two mid-length caches
        dict(name="tree t61 8k", op="tree", B=2, T=61, Hq=32, Hkv=8, d=128, lo=7001, hi=8190),
        # accumulation after a decode step over the decode workload's caches, uneven lengths
        dict(name="mass token 32k", op="mass", B=8, Lq=1, window=0, Hq=32, Hkv=8, d=128, lo=20001, hi=32768, decay=1.0),
        # weights of the last 64 rows of two 32k prompts (observation window before an eviction)
        dict(name="mass window 64", op="mass", B=2, Lq=32768, window=64, Hq=32, Hkv=8, d=128, lo=32768, hi=32768,
             decay=0.0),
        # every row of an 8k prompt
        dict(name="mass prompt 8k", op="mass", B=1, Lq=8192, window=0, Hq=32, Hkv=8, d=128, lo=8192, hi=8192, decay=0.0),
        # short caches of uneven length, d = 64: latency
        dict(name="evict short", op="evict", B=3, Hkv=2, d=64, lo=200, hi=700, keep=257, sink=4, recent=33),
        # the decode workload's caches, 32k down to 4k
        dict(name="evict 32k to 4k", op="evict", B=8, Hkv=8, d=128, lo=30000, hi=32768, keep=4096, sink=4, recent=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "tree", "mass", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 7, 8]) if op != "evict" else 1
    Hq = Hkv * G
    B = _log(rng, 1, 16)
    if op == "append":
        L = _log(rng, 1, 8192 // B)
        return dict(op=op, B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, rot=16 * rng.randint(1, d // 16),
                    layout=rng.choice(["half", "pairs"]), norm=rng.random() < 0.6, axes=rng.choice([1, 1, 3]),
                    base=rng.choice([1e4, 5e5, 1e6]), stretch=rng.choice([1.0, 4.0, 8.0]),
                    factor=rng.choice([1.0, 1.1]), far=_log(rng, 1, 2000000), cap=L + rng.randint(0, 500),
                    ragged=rng.random() < 0.5)
    if op == "tree":
        T = _log(rng, 1, 100)
        hi = max(2, min(_log(rng, 20, 32000), 2000000 // (B * T)))
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, lo=rng.randint(0, hi), hi=hi)
    if op == "mass":
        if rng.random() < 0.5:  # a few new rows over long caches
            Lq, hi = rng.randint(1, 12), _log(rng, 20, 32000)
            window = 0
        else:  # a prompt, or its last rows
            Lq = _log(rng, 20, 8000)
            hi = Lq + rng.choice([0, 0, rng.randint(1, 500)])
            window = rng.choice([0, min(Lq, _log(rng, 8, 128))])
            B = 1 if Lq > 2000 else min(B, 4)
        return dict(op=op, B=B, Lq=Lq, window=window, Hq=Hq, Hkv=Hkv, d=d, lo=max(Lq, hi // 2), hi=hi,
                    decay=rng.choice([0.0, 0.9, 1.0]))
    hi = _log(rng, 30, 131072 // B)
    keep = _log(rng, 8, hi)
    sink = rng.randint(0, keep // 4)
    return dict(op=op, B=B, Hkv=Hkv, d=d, lo=max(1, hi // 2), hi=hi, keep=keep, sink=sink,
                recent=rng.randint(0, (keep - sink) // 2))


# ------------------------------------------------------------------ the inputs

def _lens(case):
    """Lengths of the sequences: spread evenly over [lo, hi], the longest not first."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    v = [hi - (hi - lo) * b // max(1, B - 1) for b in range(B)]
    return v[1::2] + v[0::2]


def _counts(case):
    B, L = case["B"], case["L"]
    return [max(0, L - (L * b) // (B + 1)) if case["ragged"] else L for b in range(B)]


def _inv_freq(case):
    """Radians a position for each pair, an array of 64-bit floats: base^(-2p/rot), the slow half divided by `stretch`."""
    n = case["rot"] // 2
    p = torch.arange(n, dtype=torch.float64)
    f = case["base"] ** (-p / n)
    return torch.where(p >= n // 2, f / case["stretch"], f)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if case["op"] == "append":
        L, Hq, A = case["L"], case["Hq"], case["axes"]
        s = dict(case=case, qkv=_randn(g, B, L, Hq + 2 * Hkv, d))  # the output of one projection
        s["q"], s["k"], s["v"] = s["qkv"].split([Hq, Hkv, Hkv], dim=2)
        s["wq"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
        s["wk"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
        i = torch.arange(L, device=DEV)
        jitter = torch.randint(0, 50, (B, 1, 1), generator=g, device=DEV)
        if A == 1:
            pos = i[None, :, None] + case["far"] + jitter
        else:  # frames of 45 x 80 patches
            pos = torch.stack([i // 3600, i // 80 % 45, i % 80], -1)[None] + jitter
        s["pos"] = pos.to(torch.int32).contiguous()
        n = case["rot"] // 2
        s["inv_freq"] = _inv_freq(case)
        s["axis"] = (torch.arange(n) * A // n).to(torch.int32) if A > 1 else None
        s["count"] = i32(_counts(case)) if case["ragged"] else None
        s["start"] = i32([(case["cap"] - L) * (b + 1) // B for b in range(B)])
        s["k_cache"] = torch.zeros(B, case["cap"], Hkv, d, device=DEV, dtype=torch.bfloat16)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["q_out"] = torch.zeros(B, L, Hq, d, device=DEV, dtype=torch.bfloat16)
        return s
    lens = _lens(case)
    if case["op"] == "tree":
        T, Hq = case["T"], case["Hq"]
        cap = case["hi"] + T
        q, k, v = _randn(g, B, T, Hq, d), _randn(g, B, cap, Hkv, d), _randn(g, B, cap, Hkv, d)
        u = torch.nn.functional.normalize(torch.randn(d, generator=g, device=DEV), dim=0)
        q += (3 * u).to(q.dtype)
        k[:, :4] += (3 * u).to(k.dtype)
        r = np.random.RandomState(int(seed) % (1 << 31))
        words = np.zeros((B, T, -(-T // 32)), np.uint32)
        for b in range(B):
            for t in range(T):  # a node's row is its parent's and itself; parents are recent nodes, so that branches form
                if t:
                    words[b, t] = words[b, max(0, t - 1 - int(r.randint(0, 6)))]
                words[b, t, t >> 5] |= np.uint32(1 << (t & 31))
        mask = torch.from_numpy(words.view(np.int32)).to(DEV)
        return dict(case=case, q=q, k=k, v=v, lens=i32(lens), mask=mask)
    if case["op"] == "mass":
        Lq, Hq = case["Lq"], case["Hq"]
        cap = case["hi"]
        q, k = _randn(g, B, Lq, Hq, d), _randn(g, B, cap, Hkv, d)
        u = torch.nn.functional.normalize(torch.randn(d, generator=g, device=DEV), dim=0)
        q += (3 * u).to(q.dtype)
        k[:, :4] += (3 * u).to(k.dtype)
        W = case["window"] or Lq
        lse = torch.zeros(B, Hq, Lq, device=DEV)  # what the attention before it returned, for the rows that count
        for b in range(B):
            for h in range(Hq):
                x = q[b, Lq - W:, h].float() @ k[b, :lens[b], h // (Hq // Hkv)].float().T * d ** -0.5
                i = torch.arange(Lq - W, Lq, device=DEV)[:, None] + lens[b] - Lq
                x.masked_fill_(torch.arange(lens[b], device=DEV)[None] > i, float("-inf"))
                lse[b, h, Lq - W:] = torch.logsumexp(x, -1)
        mass = torch.rand(B, Hkv, cap, generator=g, device=DEV).square() if case["decay"] else None
        return dict(case=case, q=q, k=k, lse=lse, lens=i32(lens), mass=mass)
    cap, keep = case["hi"], case["keep"]
    # a few keys hold most of the weight, many hold none at all (equal: zero)
    mass = torch.exp(2 * torch.randn(B, Hkv, cap, generator=g, device=DEV) - 3)
    mass = mass * (torch.rand(B, Hkv, cap, generator=g, device=DEV) < 0.9)
    k, v = _randn(g, B, cap, Hkv, d), _randn(g, B, cap, Hkv, d)
    zeros = torch.zeros(B, keep + 64, Hkv, d, device=DEV, dtype=torch.bfloat16)  # the small cache, with room for new tokens
    return dict(case=case, k=k, v=v, mass=mass, lens=i32(lens), k_out=zeros, v_out=zeros.clone())


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        from softmax_ssa_fwd_b200 import cache
        if case["op"] == "append":
            q = cache.append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pos"], inv_freq=s["inv_freq"],
                             axis=s["axis"], interleaved=case["layout"] == "pairs", factor=case["factor"],
                             q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, start=s["start"], count=s["count"],
                             out=s["q_out"])
            return [q, s["k_cache"], s["v_cache"]]
        if case["op"] == "tree":
            return list(cache.decode_tree(s["q"], s["k"], s["v"], s["lens"], s["mask"]))
        if case["op"] == "mass":
            return [cache.attn_mass(s["q"], s["k"], s["lse"], lens=s["lens"], window=case["window"], mass=s["mass"],
                                    decay=case["decay"])]
        return list(cache.evict(s["k"], s["v"], s["mass"], s["lens"], keep=case["keep"], sink=case["sink"],
                                recent=case["recent"], k_out=s["k_out"], v_out=s["v_out"]))
    return {"append": _append, "tree": _tree, "mass": _mass, "evict": _evict}[case["op"]](s)


def _turn(x, cos, sin, case):
    """The rotation of the first `rot` columns of x [B, L, H, d]; cos, sin [B, L, 1, rot / 2]."""
    rot = case["rot"]
    t = x[..., :rot]
    if case["layout"] == "half":
        a, b = t[..., :rot // 2], t[..., rot // 2:]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([t, x[..., rot:]], -1)


def _append(s):
    case = s["case"]
    B, L = case["B"], case["L"]
    pos = s["pos"].double()
    if s["axis"] is not None:
        pos = pos[..., s["axis"].to(DEV, non_blocking=True).long()]
    t = (pos * s["inv_freq"].to(DEV, non_blocking=True))[:, :, None]
    cos, sin = (case["factor"] * torch.cos(t)).float(), (case["factor"] * torch.sin(t)).float()
    done = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        done.append(_turn(x, cos, sin, case).to(torch.bfloat16))
    q, k = done
    i = torch.arange(L, device=DEV)[None]
    rows = s["start"].long()[:, None] + i
    at = torch.arange(B, device=DEV)[:, None]
    v = s["v"]
    if s["count"] is not None:
        live = (i < s["count"][:, None])[..., None, None]
        q = torch.where(live, q, s["q_out"])
        k, v = torch.where(live, k, s["k_cache"][at, rows]), torch.where(live, v, s["v_cache"][at, rows])
    s["q_out"].copy_(q)
    s["k_cache"][at, rows] = k
    s["v_cache"][at, rows] = v
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _tree(s):
    q, k, v, lens = s["q"], s["k"], s["v"], s["lens"].long()
    B, T, Hq, d = q.shape
    cap, Hkv = k.shape[1], k.shape[2]
    x = q.float().view(B, T, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)  # rows (g, t)
    x = x @ k.float().permute(0, 2, 3, 1) * d ** -0.5
    t = torch.arange(cap, device=DEV)[None] - lens[:, None]  # the draft's number of each cache row, negative before it
    c = t.clamp(0, T - 1)[:, None].expand(B, T, cap)
    bit = (s["mask"].gather(2, c >> 5) >> (c & 31).int()) & 1
    sees = (t < 0)[:, None] | ((t < T)[:, None] & (bit == 1))
    x = x.view(B, Hkv, -1, T, cap).masked_fill(~sees[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)  # noqa: E741
    o = (p.view(B, Hkv, -1, cap) @ v.float().permute(0, 2, 1, 3)).view(B, Hkv, -1, T, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d).to(torch.bfloat16)
    return [o, (m + torch.log(l)).view(B, Hq, T)]


def _mass(s):
    case, k, lens = s["case"], s["k"], s["lens"].long()
    B, cap, Hkv, d = k.shape
    Lq, Hq = case["Lq"], case["Hq"]
    W = case["window"] or Lq
    q = s["q"][:, Lq - W:].float().view(B, W, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    x = (q @ k.float().permute(0, 2, 3, 1)).view(B, Hkv, -1, W, cap) * d ** -0.5
    x = torch.exp(x - s["lse"][:, :, Lq - W:].reshape(B, Hkv, -1, W, 1))
    i = torch.arange(Lq - W, Lq, device=DEV)[None] + lens[:, None] - Lq  # each row's own position
    j = torch.arange(cap, device=DEV)[None, None]
    x = x.masked_fill((j > i[..., None])[:, None, None], 0.0).sum((2, 3))
    if s["mass"] is not None:
        x = x + case["decay"] * s["mass"]
    return [x.masked_fill((j >= lens[:, None, None]), 0.0)]


def _evict(s):
    case, mass, lens = s["case"], s["mass"], s["lens"].long()
    B, Hkv, cap = mass.shape
    keep = case["keep"]
    j, n = torch.arange(cap, device=DEV)[None, None], lens[:, None, None]
    rank = torch.where((j < case["sink"]) | (j >= n - case["recent"]), torch.full_like(mass, float("inf")), mass)
    rank = torch.where(j < n, rank, torch.full_like(mass, float("-inf")))
    idx = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    live = torch.arange(keep, device=DEV)[None, None] < n
    idx = torch.sort(torch.where(live, idx, torch.full_like(idx, cap)), -1).values
    at = idx.clamp(max=cap - 1)
    b, h = torch.arange(B, device=DEV)[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None]
    for src, dst in ((s["k"], s["k_out"]), (s["v"], s["v_out"])):
        rows = src[b, at, h].permute(0, 2, 1, 3)
        dst[:, :keep] = torch.where(live.permute(0, 2, 1)[..., None], rows, dst[:, :keep])
    kept = torch.zeros(B, Hkv, s["k_out"].shape[1], device=DEV)
    kept[..., :keep] = torch.where(live, mass.gather(2, at), kept[..., :keep])
    index = torch.where(live, idx, torch.full_like(idx, -1)).int()
    return [s["k_out"], s["v_out"], kept, index, lens.clamp(max=keep).int()]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] == "append":
        n = sum(_counts(case))
        H = case["Hq"] + Hkv
        return dict(bytes=n * ((H + Hkv) * d * 4 + 4 * case["axes"]) + (8 * d if case["norm"] else 0),
                    flops=n * H * (3 * case["rot"] + (4 * d if case["norm"] else 0)))
    lens = _lens(case)
    if case["op"] == "tree":
        T, Hq = case["T"], case["Hq"]
        rows = sum(n + T for n in lens)
        return dict(bytes=rows * Hkv * d * 4 + B * T * Hq * (4 * d + 4) + B * T * 4 * (-(-T // 32)),
                    flops=4 * d * Hq * T * sum(lens) + 2 * d * Hq * T * T * B)
    if case["op"] == "mass":
        Hq = case["Hq"]
        W = case["window"] or case["Lq"]
        pairs = sum(W * n - W * (W - 1) // 2 for n in lens)
        return dict(bytes=sum(lens) * Hkv * (2 * d + (8 if case["decay"] else 4)) + B * W * Hq * (2 * d + 4),
                    flops=pairs * Hq * (2 * d + 3))
    kept = sum(min(n, case["keep"]) for n in lens) * Hkv
    return dict(bytes=sum(lens) * Hkv * 4 + kept * (8 * d + 12), flops=sum(lens) * Hkv)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _append64, "tree": _tree64, "mass": _mass64, "evict": _evict64}[case["op"]](s)


def _append64(s):
    """Pairs as complex numbers, one head at a time."""
    case = s["case"]
    B, L, Hq, d = s["q_out"].shape
    n = case["rot"] // 2
    f64 = dict(dtype=torch.float64, device=DEV)
    out = torch.zeros(B, L, Hq, d, **f64)
    kc, vc = torch.zeros(s["k_cache"].shape, **f64), torch.zeros(s["k_cache"].shape, **f64)
    freq = s["inv_freq"].tolist()
    a = list(range(n)) if case["layout"] == "half" else list(range(0, 2 * n, 2))
    c = [x + n for x in a] if case["layout"] == "half" else [x + 1 for x in a]
    counts, starts = _counts(case), s["start"].tolist()
    for b in range(B):
        m, at = counts[b], starts[b]
        p = s["pos"][b, :m].double()
        z = torch.empty(m, n, dtype=torch.complex128, device=DEV)
        for i in range(n):
            t = p[:, int(s["axis"][i]) if s["axis"] is not None else 0] * freq[i]
            z[:, i] = torch.polar(torch.full_like(t, case["factor"]), t)
        for h in range(Hq + case["Hkv"]):
            isq = h < Hq
            x = (s["q"][b, :m, h] if isq else s["k"][b, :m, h - Hq]).double()
            w = s["wq"] if isq else s["wk"]
            if w is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * w.double()
            y = torch.complex(x[:, a], x[:, c]) * z
            x[:, a], x[:, c] = y.real, y.imag
            if isq:
                out[b, :m, h] = x
            else:
                kc[b, at:at + m, h - Hq] = x
        vc[b, at:at + m] = s["v"][b, :m].double()
    return [out, kc, vc]


def _tree64(s):
    q, k, v, lens = s["q"], s["k"], s["v"], s["lens"].tolist()
    B, T, Hq, d = q.shape
    G = Hq // k.shape[2]
    words = s["mask"].cpu().numpy().view(np.uint32)
    out = torch.zeros(B, T, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Hq, T, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = lens[b]
        hide = np.array([[not (int(words[b, i, t // 32]) >> (t % 32)) & 1 for t in range(T)] for i in range(T)])
        hide = torch.from_numpy(hide).to(DEV)
        for h in range(k.shape[2]):
            kk, vv = k[b, :n + T, h].double(), v[b, :n + T, h].double()
            x = torch.einsum("tgd,jd->gtj", q[b, :, h * G:(h + 1) * G].double(), kk) / math.sqrt(d)
            x[:, :, n:].masked_fill_(hide, float("-inf"))
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("gtj,jd->tgd", torch.softmax(x, -1), vv)
    return [out, lse]


def _mass64(s):
    case, q, k, lens = s["case"], s["q"], s["k"], s["lens"].tolist()
    B, cap, Hkv, d = k.shape
    Lq, G = case["Lq"], case["Hq"] // Hkv
    first = Lq - (case["window"] or Lq)
    out = torch.zeros(B, Hkv, cap, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = lens[b]
        for h in range(Hkv):
            total = torch.zeros(n, dtype=torch.float64, device=DEV)
            for hq in range(h * G, (h + 1) * G):
                x = q[b, first:, hq].double() @ k[b, :n, h].double().T / math.sqrt(d)
                w = torch.exp(x - s["lse"][b, hq, first:, None].double())
                total += torch.tril(w, diagonal=n - Lq + first).sum(0)
            if s["mass"] is not None:
                total += case["decay"] * s["mass"][b, h, :n].double()
            out[b, h, :n] = total
    return [out]


def _evict64(s):
    case, lens = s["case"], s["lens"].tolist()
    B, Hkv, cap = s["mass"].shape
    keep, sink, recent = case["keep"], case["sink"], case["recent"]
    mass = s["mass"].cpu().numpy()
    ko, vo = torch.zeros_like(s["k_out"]), torch.zeros_like(s["v_out"])
    mo = np.zeros((B, Hkv, ko.shape[1]), np.float64)
    index = np.full((B, Hkv, keep), -1, np.int32)
    for b in range(B):
        n = lens[b]
        for h in range(Hkv):
            if n <= keep:
                at = np.arange(n)
            else:
                mid = np.arange(sink, n - recent)
                best = mid[np.lexsort((mid, -mass[b, h, mid]))][:keep - sink - recent]
                at = np.concatenate([np.arange(sink), np.sort(best), np.arange(n - recent, n)])
            index[b, h, :len(at)] = at
            mo[b, h, :len(at)] = mass[b, h, at]
            rows = torch.from_numpy(at).to(DEV)
            ko[b, :len(at), h], vo[b, :len(at), h] = s["k"][b, rows, h], s["v"][b, rows, h]
    return [ko.double(), vo.double(), mo, index, np.array([min(n, keep) for n in lens], np.int32)]
