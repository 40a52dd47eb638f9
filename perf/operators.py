"""Measured cases of the serving operators around block-sparse attention.

Four operators: rotary positions (with the append of new tokens to a KV cache, and
their gradient), attention of a tree of drafted tokens over the kept blocks of a
cache, the attention weight that every cached key has accumulated, and the eviction
of the keys with the least of it. ``run`` computes them in plain torch operations, or
with ``own`` set by the library's calls; ``exact`` from their definitions in fp64.

Sizes are those of the repository's workloads (32/8 heads of 128 features, caches and
prompts of 1000 to 131072 tokens, blocks of 16 to 128 keys) and generic ones between.
"""
import math

import numpy as np
import torch

own = False



def listed():
    return [
        # one decode step of 16 sequences of different lengths: rotate the new query and
        # key, append key and value to the cache (latency is all of it)
        dict(name="rope decode step", op="append", dtype="bf16", B=16, Hq=32, Hkv=8, L=1, T=4096, d=128,
             rot=128, layout="half", scaling="none", ragged=True),
        # a 32K prompt: Q and K of a fused projection rotated into the attention's layout,
        # positions scaled beyond the trained length
        dict(name="rope prefill 32K", op="rope", dtype="bf16", B=1, Hq=32, Hkv=8, L=32768, d=128, rot=128,
             layout="half", scaling="parts", backward=False, packed=True),
        # the gradient in fp32, half of each head rotated, interleaved pairs, odd length
        dict(name="rope gradient fp32", op="rope", dtype="f32", B=1, Hq=4, Hkv=2, L=700, d=128, rot=64,
             layout="interleaved", scaling="linear", backward=True, packed=False),
        # a small tree on short caches: three sequences, seven nodes, blocks of 16
        dict(name="tree 7 nodes T 1000", op="tree", B=3, Hq=8, Hkv=2, n=7, T=1000, block=16, kept=0.8,
             ragged=False),
        # 16 drafted tokens over four 128K caches, half of the blocks kept
        dict(name="tree 16 nodes 128K", op="tree", B=4, Hq=32, Hkv=8, n=16, T=131072, block=16, kept=0.5,
             ragged=False),
        # 64 drafted tokens over one 32K cache, blocks of 128
        dict(name="tree 64 nodes 32K", op="tree", B=1, Hq=32, Hkv=8, n=64, T=32768, block=128, kept=0.75,
             ragged=False),
        # eight sequences of different lengths, every block read, five heads per kv-head,
        # trees of different sizes padded to 33
        dict(name="tree 33 nodes ragged", op="tree", B=8, Hq=40, Hkv=8, n=33, T=16000, block=64, kept=0.0,
             ragged=True),
        # the weight one decode step adds, over the kept blocks of four 128K caches
        dict(name="weight decode 128K", op="weight", B=4, Hq=32, Hkv=8, Lq=1, T=131072, block=16, kept=0.75,
             ragged=False, prev=True),
        # the weight that the last 128 queries of a 32K prompt give every key
        dict(name="weight window 32K", op="weight", B=1, Hq=32, Hkv=8, Lq=128, T=32768, block=128, kept=0.0,
             ragged=False, prev=False),
        # all queries of a 4K prompt (causal: half of the square)
        dict(name="weight all of 4K", op="weight", B=1, Hq=32, Hkv=8, Lq=4096, T=4096, block=128, kept=0.0,
             ragged=False, prev=False),
        # a 32K prompt cut to 4096 keys per kv-head
        dict(name="evict 32K to 4K", op="evict", dtype="bf16", B=1, Hkv=8, T=32768, n_keep=4096, n_sink=4,
             n_recent=128, d=128, ragged=False),
        # 16 sequences in flight, of different lengths, cut to 1000 keys
        dict(name="evict 16 ragged to 1000", op="evict", dtype="bf16", B=16, Hkv=8, T=4000, n_keep=1000,
             n_sink=4, n_recent=64, d=128, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "rope", "tree", "weight", "evict"))
    G, Hkv = rng.choice((1, 2, 4, 5, 8)), rng.choice((1, 2, 4, 8))
    if op == "append":
        L = rng.choice((1, rng.randint(2, 64)))
        d = rng.choice((64, 128))
        return dict(op=op, dtype=rng.choice(("bf16", "f32")), B=_log(rng, 1, 32), Hq=G * Hkv, Hkv=Hkv, L=L,
                    T=L + _log(rng, 100, 4000), d=d, rot=rng.choice((d, d // 2)),
                    layout=rng.choice(("half", "interleaved")), scaling=rng.choice(("none", "linear", "ntk", "parts")),
                    ragged=True)
    if op == "rope":
        d = rng.choice((64, 128))
        return dict(op=op, dtype=rng.choice(("bf16", "f32")), B=rng.randint(1, 3), Hq=G * Hkv, Hkv=Hkv,
                    L=_log(rng, 1, 8000), d=d, rot=rng.choice((d, d, d // 2, 24)),
                    layout=rng.choice(("half", "interleaved")), scaling=rng.choice(("none", "linear", "ntk", "parts")),
                    backward=rng.random() < 0.5, packed=rng.random() < 0.5)
    if op == "tree":
        n = _log(rng, 1, 128)
        T = n + _log(rng, 1, 40000)
        kept = rng.choice((0.0, rng.uniform(0.05, 1.0)))
        B = max(1, min(rng.randint(1, 12), int(4e9 / (T * n * G * Hkv * 4)), int(400000 / T) + 1))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, n=n, T=T, block=rng.choice((16, 32, 64, 128)), kept=kept,
                    ragged=rng.random() < 0.5)
    if op == "weight":
        T = _log(rng, 1, 40000)
        Lq = min(T, rng.choice((1, _log(rng, 1, 512), _log(rng, 1, 3000))))
        kept = rng.choice((0.0, rng.uniform(0.1, 1.0))) if Lq == 1 else 0.0
        B = max(1, min(rng.randint(1, 12), int(2e9 / (T * Lq * G * Hkv * 4)), int(200000 / T) + 1))
        if B * G * Hkv * Lq * T > 1 << 30:
            Lq = max(1, (1 << 30) // (B * G * Hkv * T))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, Lq=Lq, T=T, block=rng.choice((16, 32, 64, 128)), kept=kept,
                    ragged=rng.random() < 0.5, prev=rng.random() < 0.5)
    T = _log(rng, 64, 40000)
    keep = _log(rng, 2, T)
    sink = rng.randint(0, min(8, keep))
    return dict(op=op, dtype=rng.choice(("bf16", "f32")), B=max(1, min(rng.randint(1, 12), 100000 // T)), Hkv=Hkv, T=T,
                n_keep=keep, n_sink=sink, n_recent=rng.randint(0, min(128, keep - sink)), d=rng.choice((64, 128)),
                ragged=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _lists(g, B, Hq, Hkv, nb, kept):
    """Ascending kept lists: the kv-head's blocks (first and last among them) are all
    kept by the group's first head and seven eighths of them by each other head."""
    G = Hq // Hkv
    m = max(min(2, nb), round(kept * nb))
    r = torch.rand(B, Hkv, nb, generator=g, device="cuda")
    r[..., 0] = r[..., nb - 1] = 2.0
    base = torch.zeros(B, Hkv, nb, dtype=torch.bool, device="cuda")
    base.scatter_(2, r.topk(m, dim=2).indices, True)
    own_ = torch.rand(B, Hkv, G, nb, generator=g, device="cuda") > 0.125
    own_[:, :, 0] = True
    own_[..., 0] = own_[..., nb - 1] = True
    keep = (base[:, :, None] & own_).reshape(B, Hq, 1, nb)
    j = torch.arange(nb, device="cuda", dtype=torch.int32)
    idx = torch.where(keep, j, torch.full_like(j, nb)).sort(dim=3).values
    return idx.to(torch.int32).contiguous(), keep.sum(3).to(torch.int32).contiguous()


def _freqs(case):
    """Radians per position of each pair, and the factor on the rotated values."""
    rot, base, factor, trained = case["rot"], 10000.0, 4.0, 8192
    c = np.arange(rot // 2, dtype=np.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * c / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":
        # pairs that turn more than 32 times in the trained length are kept, those that
        # turn less than once are interpolated, with a ramp between
        def at(turns):
            return rot * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = np.clip((c - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        f = f * (1.0 - ramp) + f / factor * ramp
        return f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, dt = case["op"], case["B"], _dtype(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    s = dict(case=case, op=op)
    if op in ("append", "rope"):
        Hq, Hkv, L, d = case["Hq"], case["Hkv"], case["L"], case["d"]
        freqs, s["mscale"] = _freqs(case)
        s["freqs"] = torch.from_numpy(freqs)
        if op == "append" or case["packed"]:
            qkv = randn(B, L, Hq + 2 * Hkv, d).transpose(1, 2)     # the fused projection's output
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["q"], s["k"] = randn(B, Hq, L, d), randn(B, Hkv, L, d)
        if op == "append":
            T = case["T"]
            s["kc"], s["vc"] = randn(B, Hkv, T, d), randn(B, Hkv, T, d)
            s["rows"] = torch.randint(0, T - L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            s["pos"] = (s["rows"][:, None] + torch.arange(L, device="cuda", dtype=torch.int32)).contiguous()
        else:
            s["pos"] = None
        return s
    Hkv, T, d = case["Hkv"], case["T"], case.get("d", 128)
    s["kc"] = randn(B, Hkv, T, d)
    if op == "evict":
        s["vc"] = randn(B, Hkv, T, d)
        # accumulated softmax weight: heavy-tailed, many keys with next to none (equal)
        s["score"] = torch.rand(B, Hkv, T, generator=g, device="cuda").pow(8).mul(1e4).round().div(1e4)
        s["lens"] = None
        if case["ragged"]:
            s["lens"] = torch.randint(1, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        # the smaller cache that the kept rows move to; rows that no key fills stay zero
        for name in ("kc", "vc"):
            s[name + "_out"] = torch.zeros(B, Hkv, case["n_keep"], d, device="cuda", dtype=dt)
        s["score_out"] = torch.zeros(B, Hkv, case["n_keep"], device="cuda")
        return s
    Hq = case["Hq"]
    nb = -(-T // case["block"])
    s["scale"] = float(np.float32(1.0 / math.sqrt(d)))
    s["idx"] = s["count"] = s["lens"] = None
    if case["kept"] > 0:
        s["idx"], s["count"] = _lists(g, B, Hq, Hkv, nb, case["kept"])
    if op == "tree":
        n = case["n"]
        s["vc"] = randn(B, Hkv, T, d)
        s["q"] = randn(B, Hq, n, d)
        i = torch.arange(n, device="cuda")
        parents = (torch.rand(B, n, generator=g, device="cuda") * i).floor().long().clamp(max=n - 1)
        parents[:, 0] = -1
        if case["ragged"]:
            s["lens"] = torch.randint(0, T - n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            size = torch.randint(max(1, n // 2), n + 1, (B, 1), generator=g, device="cuda")
            parents = torch.where(i < size, parents, -2)         # unused nodes of smaller trees
        s["parents"] = parents.to(torch.int32)
        return s
    Lq = case["Lq"]
    s["q"] = randn(B, Hq, Lq, d)
    if case["ragged"]:
        s["lens"] = torch.randint(Lq, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    s["prev"] = torch.rand(B, Hkv, T, generator=g, device="cuda") if case["prev"] else None
    ok = _visible(s)
    x = _scores(s["q"], s["kc"], s["scale"])
    s["lse"] = x.masked_fill_(~ok, -math.inf).logsumexp(-1)       # attention's log-sum-exp
    return s


# ---------------------------------------------------------------- plain forms

def _scores(q, k, scale):
    B, Hq, n, d = q.shape
    G = Hq // k.shape[1]
    x = q.float().reshape(B, Hq // G, G * n, d) @ k.float().transpose(2, 3)
    return (x * scale).reshape(B, Hq, n, -1)


def _kept(idx, count, T, block):
    """[B, Hq, 1, T]: whether the key's block is on the head's list."""
    nb, cap = -(-T // block), idx.shape[3]
    at = torch.arange(cap, device=idx.device) < count[..., None]
    on = torch.zeros(*idx.shape[:3], nb + 1, dtype=torch.bool, device=idx.device)
    on.scatter_(3, torch.where(at, idx, nb).long(), at)
    return on[..., torch.arange(T, device=idx.device) // block]


def _visible(s):
    """Which keys the queries at the sequence's end see: [B, Hq or 1, Lq, T]."""
    B, Hq, Lq, _ = s["q"].shape
    T = s["kc"].shape[2]
    t = torch.arange(T, device="cuda")
    n = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device="cuda")
    at = n[:, None] - Lq + torch.arange(Lq, device="cuda")
    ok = (t <= at[..., None])[:, None]
    return ok if s["idx"] is None else ok & _kept(s["idx"], s["count"], T, s["case"]["block"])


def _rotate(x, cos, sin, rot, layout):
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((y, rest), -1)


def _plain_rope(s):
    c = s["case"]
    B, L, dt = c["B"], c["L"], _dtype(c)
    pos = s["pos"] if s["pos"] is not None else torch.arange(L, device="cuda").expand(B, L)
    ang = pos.double()[:, None, :, None] * s["freqs"].cuda()      # far positions: fp64 angles
    cos, sin = (ang.cos() * s["mscale"]).float(), (ang.sin() * s["mscale"]).float()
    if c.get("backward"):
        sin = -sin
    q = _rotate(s["q"], cos, sin, c["rot"], c["layout"]).to(dt)
    k = _rotate(s["k"], cos, sin, c["rot"], c["layout"]).to(dt)
    if c["op"] == "rope":
        return dict(q=q, k=k)
    b = torch.arange(B, device="cuda")[:, None]
    rows = s["rows"].long()[:, None] + torch.arange(L, device="cuda")
    s["kc"][b, :, rows] = k.transpose(1, 2)
    s["vc"][b, :, rows] = s["v"].transpose(1, 2)
    return dict(q=q, kc=s["kc"], vc=s["vc"])


def _plain_tree(s):
    q, kc, vc, parents = s["q"], s["kc"], s["vc"], s["parents"].long()
    B, Hq, n, d = q.shape
    Hkv, T = kc.shape[1], kc.shape[2]
    node = torch.arange(n, device="cuda")
    edge = (parents[..., None] == node).double() + torch.eye(n, device="cuda", dtype=torch.float64)
    sees = (torch.linalg.matrix_power(edge, n) > 0) & (parents >= -1)[..., None]    # ancestors and itself
    P = s["lens"].long() if s["lens"] is not None else torch.full((B,), T - n, device="cuda")
    t = torch.arange(T, device="cuda")
    old = (t < P[:, None])[:, None, None] & (parents >= -1)[:, None, :, None]
    if s["idx"] is not None:
        old = old & _kept(s["idx"], s["count"], T, s["case"]["block"])
    off = t - P[:, None]
    drafted = sees.gather(2, off.clamp(0, n - 1)[:, None].expand(B, n, T)) & ((off >= 0) & (off < n))[:, None]
    x = _scores(q, kc, s["scale"]).masked_fill_(~(old | drafted[:, None]), -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (x - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, T) @ vc.float()).reshape(B, Hq, n, d) / torch.where(l > 0, l, torch.ones_like(l))
    return dict(out=o.to(q.dtype), lse=(l.log() + m)[..., 0])


def _plain_weight(s):
    B, Hkv, T = s["kc"].shape[:3]
    x = _scores(s["q"], s["kc"], s["scale"]).sub_(s["lse"][..., None])
    w = x.exp_().mul_(_visible(s)).reshape(B, Hkv, -1, T).sum(2)
    return w if s["prev"] is None else s["prev"] + w


def _plain_evict(s):
    c, score = s["case"], s["score"]
    B, Hkv, T = score.shape
    n_keep = c["n_keep"]
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device="cuda")
    t = torch.arange(T, device="cuda")
    kind = ((t < c["n_sink"]) | (t >= lens[:, None] - c["n_recent"])).long() + 1        # 2: always kept
    kind = torch.where(t < lens[:, None], kind, 0)[:, None].expand(B, Hkv, T)           # 0: no key there
    order = score.sort(dim=2, descending=True, stable=True).indices                     # ties: the lowest index
    order = order.gather(2, kind.gather(2, order).sort(dim=2, descending=True, stable=True).indices)
    count = lens.clamp(max=n_keep).to(torch.int32)
    filled = torch.arange(n_keep, device="cuda") < count[:, None, None]
    keep = torch.where(filled, order[..., :n_keep], T).sort(dim=2).values
    row = keep.clamp(max=T - 1)
    for src, dst in ((s["kc"], s["kc_out"]), (s["vc"], s["vc_out"])):
        got = src.gather(2, row[..., None].expand(B, Hkv, n_keep, src.shape[3]))
        dst.copy_(torch.where(filled[..., None], got, dst))
    s["score_out"].copy_(torch.where(filled, score.gather(2, row), s["score_out"]))
    return dict(keep=torch.where(filled, keep, -1).to(torch.int32), count=count, k=s["kc_out"], v=s["vc_out"],
                score=s["score_out"])


# ---------------------------------------------------------------- one pass

def run(s):
    c, op = s["case"], s["op"]
    if not own:
        return dict(append=_plain_rope, rope=_plain_rope, tree=_plain_tree, weight=_plain_weight,
                    evict=_plain_evict)[op](s)
    import block_sparse_long_stats_b200 as spa
    if op == "rope":
        q, k = spa.spa_rope(s["q"], s["k"], s["freqs"], s["mscale"], layout=c["layout"], backward=c["backward"])
        return dict(q=q, k=k)
    if op == "append":
        q = spa.spa_rope_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["freqs"], s["mscale"], rows=s["rows"],
                                layout=c["layout"], pos=s["pos"])
        return dict(q=q, kc=s["kc"], vc=s["vc"])
    if op == "tree":
        out, lse = spa.spa_sparse_attn_tree(s["q"], s["kc"], s["vc"], s["parents"], c["block"], s["idx"], s["count"],
                                            s["scale"], lens=s["lens"], want_lse=True)
        return dict(out=out, lse=lse)
    if op == "weight":
        return spa.spa_attn_weight(s["q"], s["kc"], s["lse"], s["scale"], block=c["block"], idx=s["idx"],
                                   count=s["count"], lens=s["lens"], prev=s["prev"])
    keep, count = spa.spa_evict_select(s["score"], c["n_keep"], c["n_sink"], c["n_recent"], lens=s["lens"])
    k, v, score = spa.spa_cache_gather(s["kc"], s["vc"], keep, count, score=s["score"], k_out=s["kc_out"],
                                       v_out=s["vc_out"], score_out=s["score_out"])
    return dict(keep=keep, count=count, k=k, v=v, score=score)


def work(case):
    op, B = case["op"], case["B"]
    size = 4 if case.get("dtype") == "f32" else 2
    if op in ("rope", "append"):
        heads, L, d = case["Hq"] + case["Hkv"], case["L"], case["d"]
        moved = heads + (case["Hkv"] if op == "append" else 0)      # each row read once, written once
        return dict(bytes=2 * B * moved * L * d * size, flops=3 * B * heads * L * case["rot"])
    Hkv, T = case["Hkv"], case["T"]
    if op == "evict":
        d = case["d"]
        rows = min(case["n_keep"], T)
        share = 0.5 * (1 + 1.0 / T) if case["ragged"] else 1.0      # mean length over the capacity
        # scores once, kept rows of K, V and score read and written, the list written
        return dict(bytes=B * Hkv * (4 * T * share + rows * (4 * d * size + 4 + 4)), flops=B * Hkv * T)
    G = case["Hq"] // Hkv
    d = 128
    if op == "tree":
        n = case["n"]
        keys = (T - n) * (0.5 if case["ragged"] else 1.0) * (case["kept"] or 1.0) + n
        rows = B * Hkv * G * n
        return dict(bytes=B * Hkv * keys * 2 * d * 2 + rows * (2 * d * 2 + 4), flops=4 * rows * keys * d)
    Lq = case["Lq"]
    keys = (T + Lq) / 2 if case["ragged"] else T
    pairs = B * Hkv * G * (Lq * keys - Lq * (Lq - 1) / 2) * (case["kept"] or 1.0)
    return dict(bytes=B * Hkv * (keys * (case["kept"] or 1.0) * d * 2 + T * (8 if case["prev"] else 4))
                + B * Hkv * G * Lq * (d * 2 + 4), flops=2 * pairs * d)


# ---------------------------------------------------------------- definitions in fp64

def exact(case, seed):
    s = prepare(case, seed)
    op, B = case["op"], case["B"]
    if op in ("rope", "append"):
        return _exact_rope(case, s)
    if op == "evict":
        return _exact_evict(case, s)
    Hq, Hkv, T = case["Hq"], case["Hkv"], case["T"]
    G = Hq // Hkv
    rows = case["n"] if op == "tree" else case["Lq"]
    out = torch.zeros(B, Hq, rows, 128, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, rows), -math.inf, dtype=torch.float64, device="cuda")
    acc = torch.zeros(B, Hkv, T, dtype=torch.float64, device="cuda")
    if op == "weight" and s["prev"] is not None:
        acc += s["prev"]
    for b in range(B):
        length = T if op == "weight" else T - rows
        if s["lens"] is not None:
            length = int(s["lens"][b])
        if op == "tree":
            up = s["parents"][b].tolist()
            see = torch.zeros(rows, rows, dtype=torch.bool)
            for i in range(rows):
                j = i if up[i] >= -1 else -1
                while j >= 0:
                    see[i, j] = True
                    j = up[j]
            use = torch.tensor([p >= -1 for p in up], device="cuda")
        for h in range(Hq):
            # the cached keys on the head's list
            t = torch.arange(length, device="cuda")
            if s["idx"] is not None:
                blocks = s["idx"][b, h, 0, :int(s["count"][b, h, 0])]
                t = t[torch.isin(t // case["block"], blocks)]
            K, q = s["kc"][b, h // G].double(), s["q"][b, h].double()
            if op == "weight":
                x = (q @ K[t].T) * s["scale"] - s["lse"][b, h].double()[:, None]
                at = length - rows + torch.arange(rows, device="cuda")
                acc[b, h // G, t] += torch.where(t[None] <= at[:, None], x.exp(), 0.0).sum(0)
                continue
            V = s["vc"][b, h // G].double()
            t = torch.cat((t, length + torch.arange(rows, device="cuda")))
            seen = torch.cat((use[:, None].expand(rows, len(t) - rows), see.cuda()), 1)
            x = torch.where(seen, (q @ K[t].T) * s["scale"], -math.inf)
            lse[b, h] = x.logsumexp(1)
            out[b, h] = torch.where(seen, (x - lse[b, h][:, None]).exp(), 0.0) @ V[t]
    return acc if op == "weight" else dict(out=out, lse=lse)


def _exact_rope(case, s):
    B, L, rot = case["B"], case["L"], case["rot"]
    pos = np.tile(np.arange(L), (B, 1)) if s["pos"] is None else s["pos"].cpu().numpy()
    turn = np.exp(1j * pos[:, None, :, None].astype(np.float64) * s["freqs"].numpy()) * s["mscale"]
    if case.get("backward"):
        turn = turn.conj()

    def rotated(x):
        x = x.double().cpu().numpy()
        y = x.copy()
        first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half"
                         else (slice(0, rot, 2), slice(1, rot, 2)))
        z = (x[..., first] + 1j * x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return torch.from_numpy(y)

    q, k = rotated(s["q"]), rotated(s["k"])
    if case["op"] == "rope":
        return dict(q=q, k=k)
    kc, vc, rows = s["kc"].double().cpu(), s["vc"].double().cpu(), s["rows"].tolist()
    for b in range(B):
        kc[b, :, rows[b]:rows[b] + L] = k[b]
        vc[b, :, rows[b]:rows[b] + L] = s["v"][b].double().cpu()
    return dict(q=q, kc=kc, vc=vc)


def _exact_evict(case, s):
    B, Hkv, T, n_keep = case["B"], case["Hkv"], case["T"], case["n_keep"]
    score = s["score"].cpu().numpy().astype(np.float64)
    keep = np.full((B, Hkv, n_keep), -1, np.int32)
    count = np.zeros(B, np.int32)
    k, v, kept = s["kc_out"].double(), s["vc_out"].double(), s["score_out"].double()
    for b in range(B):
        length = T if s["lens"] is None else int(s["lens"][b])
        count[b] = c = min(length, n_keep)
        t = np.arange(length)
        fixed = (t < case["n_sink"]) | (t >= length - case["n_recent"])
        for g in range(Hkv):
            best = np.lexsort((t, -score[b, g, :length], ~fixed))[:c]
            keep[b, g, :c] = np.sort(best)
            row = torch.from_numpy(keep[b, g, :c].astype(np.int64)).cuda()
            k[b, g, :c], v[b, g, :c] = s["kc"][b, g, row].double(), s["vc"][b, g, row].double()
            kept[b, g, :c] = s["score"][b, g, row].double()
    return dict(keep=torch.from_numpy(keep), count=torch.from_numpy(count), k=k, v=v, score=kept)
