"""The serving operators against plain fp64 implementations: rotary positions (and their
gradient), tree attention, accumulated attention weight, eviction, and a run of them
together. Tolerances are derived beside each check: U = half a step of bf16 (2^-8,
relative) counts bf16 roundings, E = 2^-24 those of fp32."""
import math

import pytest
import torch

import block_sparse_long_stats_b200 as spa

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def ok():
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() == 0


# ---------------------------------------------------------------- rotary positions

def ref_rope(x, pos, freqs, m, layout, backward=False):
    """fp64 rotation and the magnitude its rounding errors scale with."""
    rot = 2 * len(freqs)
    x = x.double()
    a = pos.double()[:, None, :, None] * freqs.cuda()
    c, s = a.cos() * m, a.sin() * (-m if backward else m)
    y, mag = x.clone(), x.abs()
    one, two = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
                else (slice(0, rot, 2), slice(1, rot, 2)))
    x1, x2 = x[..., one], x[..., two]
    y[..., one], y[..., two] = x1 * c - x2 * s, x2 * c + x1 * s
    mag[..., one] = mag[..., two] = (x1.abs() + x2.abs()) * abs(m)
    return y, mag


def close_rope(got, want, mag, dtype):
    # sine and cosine of an angle reduced in fp64: 4 E; times mscale, products, sum: 4 E
    # more; bf16 rounds the result once
    tol = 8 * E * mag + (U * want.abs() if dtype == BF else 0.0)
    assert got.dtype == dtype and bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,B,Hq,Hkv,L,d,rot", [
    (BF, 2, 8, 2, 33, 128, 128), (BF, 1, 3, 1, 7, 128, 24), (BF, 1, 1, 1, 1, 64, 2), (BF, 1, 5, 1, 130, 96, 50),
    (F32, 2, 4, 2, 65, 128, 64), (F32, 1, 2, 1, 9, 64, 6), (BF, 1, 32, 8, 1500, 128, 128), (F32, 1, 40, 8, 600, 256, 256),
])
@pytest.mark.parametrize("packed", [False, True])
def test_rope_matches_fp64_and_its_gradient_is_the_transpose(layout, dtype, B, Hq, Hkv, L, d, rot, packed):
    g = gen(L + rot)
    if packed:      # the fused projection's output, one odd feature in front
        x = randn(g, B, L, (Hq + Hkv) * d + 1, dtype=dtype)[..., 1:].unflatten(2, (Hq + Hkv, d)).transpose(1, 2)
        q, k = x[:, :Hq], x[:, Hq:]
    else:
        q, k = randn(g, B, Hq, L, d, dtype=dtype), randn(g, B, Hkv, L, d, dtype=dtype)
    freqs, m = spa.spa_rope_frequencies(rot, 10000.0, "parts", factor=8.0, trained=4096)
    pos = torch.randint(-(1 << 20), 1 << 30, (B, L), generator=g, device="cuda", dtype=torch.int32)
    for backward in (False, True):
        a, b = spa.spa_rope(q, k, freqs, m, layout, pos=pos, backward=backward)
        for got, x in ((a, q), (b, k)):
            want, mag = ref_rope(x, pos, freqs, m, layout, backward)
            close_rope(got, want, mag, dtype)
            assert torch.equal(got[..., rot:], x[..., rot:])
    ok()


def test_rope_gradient_matches_differences():
    # the rotation is linear: <R x, w> for x and x + e_c differ by (R^T w)_c exactly
    g = gen(1)
    x, w = randn(g, 1, 1, 1, 64, dtype=F32), randn(g, 1, 1, 1, 64, dtype=F32)
    freqs, m = spa.spa_rope_frequencies(48, 10000.0, "linear", factor=2.0)
    grad, _ = spa.spa_rope(w, None, freqs, m, "interleaved", pos0=777, backward=True)
    eye = torch.eye(64, device="cuda").reshape(64, 1, 1, 64)
    moved, _ = spa.spa_rope((x + eye).contiguous(), None, freqs, m, "interleaved", pos0=777)
    base, _ = spa.spa_rope(x, None, freqs, m, "interleaved", pos0=777)
    diff = ((moved.double() - base.double()) * w.double()).sum(-1).reshape(-1)
    # |x| < 8: x + 1 and both results are rounded to 16 E, for 2 features of each pair
    assert bool(((diff - grad.double().reshape(-1)).abs() <= 2 * 64 * E * w.abs().max()).all())
    ok()


def test_rope_in_place_and_into_strided_outputs():
    g = gen(2)
    freqs, m = spa.spa_rope_frequencies(128)
    x = randn(g, 2, 9, 4, 128).transpose(1, 2)
    want, _ = spa.spa_rope(x, None, freqs, m)
    y = x.clone(memory_format=torch.preserve_format)
    out, _ = spa.spa_rope(y, None, freqs, m, q_out=y)
    assert out is y and torch.equal(y, want)
    big = torch.full((2, 4, 20, 128), 7.0, device="cuda", dtype=BF)
    spa.spa_rope(x, None, freqs, m, q_out=big[:, :, 5:14])
    assert torch.equal(big[:, :, 5:14], want) and bool((big[:, :, :5] == 7).all() and (big[:, :, 14:] == 7).all())
    ok()


@pytest.mark.parametrize("dtype,d,L", [(BF, 128, 1), (F32, 64, 5), (BF, 64, 17)])
def test_rope_append_writes_its_rows_only(dtype, d, L):
    g = gen(3)
    B, Hq, Hkv, T = 4, 6, 3, 50
    qkv = randn(g, B, L, Hq + 2 * Hkv, d, dtype=dtype).transpose(1, 2)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    freqs, m = spa.spa_rope_frequencies(d, 500.0)
    kc, vc = randn(g, B, Hkv, T, d, dtype=dtype), randn(g, B, Hkv, T, d, dtype=dtype)
    k0, v0 = kc.clone(), vc.clone()
    rows = torch.tensor([0, 20, T - L, 7], device="cuda", dtype=torch.int32)
    out = spa.spa_rope_append(q, k, v, kc, vc, freqs, m, rows=rows)
    pos = rows[:, None] + torch.arange(L, device="cuda")
    wq, mq = ref_rope(q, pos, freqs, m, "half")
    wk, mk = ref_rope(k, pos, freqs, m, "half")
    close_rope(out, wq, mq, dtype)
    for b in range(B):
        r = slice(int(rows[b]), int(rows[b]) + L)
        close_rope(kc[b, :, r], wk[b], mk[b], dtype)
        assert torch.equal(vc[b, :, r], v[b])
        k0[b, :, r], v0[b, :, r] = kc[b, :, r], vc[b, :, r]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    ok()
    one = spa.spa_rope_append(q, k, v, kc, vc, freqs, m, row0=30)
    close_rope(one, *ref_rope(q, torch.arange(30, 30 + L, device="cuda").expand(B, L), freqs, m, "half"), dtype)
    assert torch.equal(vc[:, :, 30:30 + L], v)
    ok()


def test_rope_append_skips_rows_outside_the_cache():
    g = gen(4)
    q, k, v = (randn(g, 3, 2, 4, 64) for _ in range(3))
    kc, vc = randn(g, 3, 2, 10, 64), randn(g, 3, 2, 10, 64)
    k0, v0 = kc.clone(), vc.clone()
    freqs, m = spa.spa_rope_frequencies(64)
    rows = torch.tensor([-2, 8, 2 ** 31 - 2], device="cuda", dtype=torch.int32)
    spa.spa_rope_append(q, k, v, kc, vc, freqs, m, rows=rows, pos=torch.zeros(3, 4, device="cuda", dtype=torch.int32))
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() == 1                      # SPA_DEVERR_BAD_INDEX
    k0[0, :, 0:2], v0[0, :, 0:2] = k[0, :, 2:], v[0, :, 2:]      # position 0: not turned
    k0[1, :, 8:], v0[1, :, 8:] = k[1, :, :2], v[1, :, :2]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


# ---------------------------------------------------------------- tree attention

def lists(g, B, Hq, nb, p):
    """Ascending lists, each block kept with probability p."""
    keep = torch.rand(B, Hq, 1, nb, generator=g, device="cuda") < p
    j = torch.arange(nb, device="cuda", dtype=torch.int32)
    idx = torch.where(keep, j, nb + 5).sort(dim=3).values.to(torch.int32)
    return idx.contiguous(), keep.sum(3).to(torch.int32), keep


def tree_of(g, B, n, unused=0):
    i = torch.arange(n, device="cuda")
    p = (torch.rand(B, n, generator=g, device="cuda") * (i + 1)).floor().long().clamp(max=n) - 1
    p[:, 0] = -1
    if unused:
        p[1::2, n - unused:] = -2
    return p.to(torch.int32)


def ref_tree(q, kc, vc, parents, block, keep, scale, lens):
    """out, lse and the softmax-weighted |v| (what P's rounding scales with), fp64."""
    B, Hq, n, d = q.shape
    Hkv, T = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, n, d, dtype=torch.float64, device="cuda")
    mag, lse = out.clone(), torch.full((B, Hq, n), -math.inf, dtype=torch.float64, device="cuda")
    qk = torch.zeros_like(lse)
    for b in range(B):
        P = T - n if lens is None else int(lens[b])
        up = parents[b].tolist()
        see = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):
            j, path = i, []
            while j >= 0:
                path.append(j)
                j = up[j] if up[j] < j else -2
            if j == -1:
                see[i, path] = True
        see = see.cuda()
        for h in range(Hq):
            t = torch.arange(P, device="cuda")
            if keep is not None:
                t = t[keep[b, h, 0][t // block]]
            for i in range(n):
                if not bool(see[i, i]):
                    continue
                u = torch.cat((t, P + torch.nonzero(see[i])[:, 0]))
                K, V, x = kc[b, h // G, u].double(), vc[b, h // G, u].double(), q[b, h, i].double()
                s = (K @ x) * scale
                lse[b, h, i] = s.logsumexp(0)
                p = (s - lse[b, h, i]).exp()
                out[b, h, i], mag[b, h, i] = p @ V, p @ V.abs()
                qk[b, h, i] = (K.abs() @ x.abs()).max() * scale
    return out, lse, mag, qk


def check_tree(q, kc, vc, parents, block, keep, scale, lens, got, lse):
    want, wl, mag, qk = ref_tree(q, kc, vc, parents, block, keep, scale, lens)
    # logits: up to 128 fp32 roundings of sums of |q||k|, 128 E = 2^-17 of their size;
    # P rounded to bf16 (U of each weight, U of |v|'s mean), the output once more
    d = 2.0 ** -17 * qk + 2.0 ** -18
    tol = (1.02 * U + 2 * d[..., None]) * mag + U * want.abs()
    assert bool(((got.double() - want).abs() <= tol).all()), float(((got.double() - want).abs() / tol.clamp(min=1e-30)).max())
    dead = torch.isinf(wl)
    assert bool((lse[dead] == -math.inf).all()) and bool((got[dead] == 0).all())
    assert bool(((lse.double() - wl).abs()[~dead] <= (d + 4 * E * wl.abs())[~dead]).all())


SCALE = {64: 0.125, 128: 128.0 ** -0.5}


@pytest.mark.parametrize("B,Hq,Hkv,n,T,d,block,p,ragged", [
    (1, 1, 1, 1, 1, 128, 16, None, False),            # one token, no text before it
    (1, 4, 1, 1, 2, 64, 128, 1.0, False),
    (2, 8, 2, 7, 7, 128, 16, None, False),            # a tree and nothing else
    (3, 8, 2, 7, 1000, 128, 16, 0.5, False),
    (2, 8, 8, 33, 515, 64, 32, 0.3, True),
    (2, 10, 2, 64, 900, 128, 64, None, True),
    (1, 16, 1, 127, 2000, 128, 128, 0.6, False),
    (2, 32, 2, 128, 700, 128, 16, 0.2, True),
    (1, 3, 3, 128, 260, 64, 64, 0.0, False),          # no block kept: the tree alone
    (5, 4, 4, 2, 4097, 128, 32, 0.9, True),
    (1, 8, 1, 16, 9000, 128, 16, 0.4, False),
    (1, 8, 1, 17, 6000, 64, 128, None, False),
    (40, 8, 4, 3, 150, 64, 32, 0.5, True),            # more sequences than lanes, many units a run
    (3, 16, 8, 2, 2, 128, 16, None, False),           # a tree that fills the cache
])
def test_tree_matches_fp64(B, Hq, Hkv, n, T, d, block, p, ragged):
    g = gen(T + n)
    q, kc, vc = randn(g, B, Hq, n, d), randn(g, B, Hkv, T, d), randn(g, B, Hkv, T, d)
    parents = tree_of(g, B, n, unused=n // 3 if ragged else 0)
    lens = None
    if ragged:
        lens = torch.randint(0, T - n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        lens[0] = 0
        for b in range(B):      # rows behind the tree and of unused nodes hold anything
            bad = torch.arange(T, device="cuda") >= int(lens[b]) + n
            bad[int(lens[b]):int(lens[b]) + n] |= parents[b] < -1
            kc[b, :, bad] = float("nan")
            vc[b, :, bad] = float("inf")
    idx = count = keep = None
    if p is not None:
        idx, count, keep = lists(g, B, Hq, -(-T // block), p)
    out, lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, block, idx, count, SCALE[d], lens=lens, want_lse=True)
    ok()
    check_tree(q, kc, vc, parents, block, keep, SCALE[d], lens, out, lse)
    again, _ = spa.spa_sparse_attn_tree(q, kc, vc, parents, block, idx, count, SCALE[d], lens=lens)
    assert torch.equal(again, out)


@pytest.mark.parametrize("p,block", [(0.2, 16), (0.95, 16), (0.8, 32)])
def test_tree_lists_longer_than_a_stretch(p, block):
    # 2048 rows leave few runs: each walks over several stretches of its long lists, with
    # blocks alone or side by side
    g = gen(13)
    G, n, T = 16, 128, 450000
    q, kc, vc = randn(g, 1, G, n, 128), randn(g, 1, 1, T, 128), randn(g, 1, 1, T, 128)
    parents = tree_of(g, 1, n)
    idx, count, keep = lists(g, 1, G, -(-T // block), p)
    out, lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, block, idx, count, 0.09, want_lse=True)
    ok()
    one = [0, 9]                                       # two heads: the rest is the same
    want, wl, mag, qk = ref_tree(q[:, one], kc.expand(1, 2, T, 128), vc.expand(1, 2, T, 128), parents, block,
                                 keep[:, one], 0.09, None)
    d = 2.0 ** -17 * qk + 2.0 ** -18
    assert bool(((out[:, one].double() - want).abs() <= (1.02 * U + 2 * d[..., None]) * mag + U * want.abs()).all())
    assert bool(((lse[:, one].double() - wl).abs() <= d + 4 * E * wl.abs()).all())


def test_offsets_beyond_32_bits():
    # caches of 2.3 G elements: rows at their far end
    g = gen(14)
    B, Hq, Hkv, n, T, d = 2, 8, 8, 2, 1_100_000, 128
    kc, vc = (torch.zeros(B, Hkv, T, d, device="cuda", dtype=BF) for _ in range(2))
    assert kc.numel() > 2 ** 31
    kc[1, 7].normal_(generator=g)
    vc[1, 7].normal_(generator=g)
    q, k, v = randn(g, B, Hq, n, d), randn(g, B, Hkv, n, d), randn(g, B, Hkv, n, d)
    freqs, m = spa.spa_rope_frequencies(d)
    qr = spa.spa_rope_append(q, k, v, kc, vc, freqs, m, row0=T - n)
    pos = torch.arange(T - n, T, device="cuda").expand(B, n)
    want, mag = ref_rope(k, pos, freqs, m, "half")
    close_rope(kc[:, :, T - n:], want, mag, BF)
    assert torch.equal(vc[:, :, T - n:], v)
    parents = torch.tensor([[-1, 0]] * B, device="cuda", dtype=torch.int32)
    out, lse = spa.spa_sparse_attn_tree(qr, kc, vc, parents, 64, None, None, 0.09, want_lse=True)
    last = qr[:, :, 1:].contiguous()
    w = spa.spa_attn_weight(last, kc, lse[:, :, 1:].contiguous(), 0.09)
    keep, count = spa.spa_evict_select(w, 50, 4, 4)
    k2, v2, _ = spa.spa_cache_gather(kc, vc, keep, count)
    ok()
    check_tree(qr[1:, 7:], kc[1:, 7:], vc[1:, 7:], parents[1:], 64, None, 0.09, None, out[1:, 7:], lse[1:, 7:])
    ww, tol = ref_weight(last[1:, 7:], kc[1:, 7:], lse[1:, 7:, 1:], 0.09, 64, None, None, None, 1.0)
    assert bool(((w[1:, 7:].double() - ww).abs() <= tol).all())
    assert keep[1, 7, -4:].tolist() == list(range(T - 4, T))
    assert torch.equal(k2[1, 7], kc[1, 7, keep[1, 7].long()]) and torch.equal(v2[1, 7], vc[1, 7, keep[1, 7].long()])


def test_two_calls_at_once_on_two_streams():
    g = gen(15)
    args = []
    for T in (3000, 5000):
        q, kc, vc = randn(g, 1, 8, 20, 128), randn(g, 1, 2, T, 128), randn(g, 1, 2, T, 128)
        args.append((q, kc, vc, tree_of(g, 1, 20), 64, None, None, 0.09))
    want = [spa.spa_sparse_attn_tree(*a, want_lse=True) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(20):
        got = [spa.spa_sparse_attn_tree(*a, want_lse=True, stream=st) for a, st in zip(args, streams)]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    ok()


def test_tree_of_large_logits():
    # logits of some hundreds: the running maximum moves far between tiles
    g = gen(8)
    q, kc, vc = randn(g, 1, 4, 5, 128) * 12, randn(g, 1, 1, 3001, 128), randn(g, 1, 1, 3001, 128)
    kc *= torch.linspace(0.1, 4.0, 3001, device="cuda").to(BF)[:, None]
    parents = tree_of(g, 1, 5)
    out, lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, 64, None, None, 0.09, want_lse=True)
    ok()
    check_tree(q, kc, vc, parents, 64, None, 0.09, None, out, lse)


def test_tree_bad_parents_lists_and_lengths_are_recorded():
    g = gen(9)
    B, n, T, block = 2, 6, 400, 32
    q, kc, vc = randn(g, B, 4, n, 128), randn(g, B, 2, T, 128), randn(g, B, 2, T, 128)
    parents = torch.tensor([[-1, 0, 2, 2, 9, 1], [-1, 0, 0, -5, 3, 2]], device="cuda", dtype=torch.int32)
    idx, count, keep = lists(g, B, 4, 13, 0.6)
    out, lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, block, idx, count, 0.1, want_lse=True)
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() == 1
    # nodes 2 (its own parent) and 4 (a later one) are unused, and so is node 3, below 2
    check_tree(q, kc, vc, parents, block, keep, 0.1, None, out, lse)
    assert bool(torch.isinf(lse[0, :, 2:5]).all()) and bool(torch.isinf(lse[1, :, 3:5]).all())
    parents = tree_of(g, B, n)
    broken = torch.full((B, 4, 1, 20), 99, device="cuda", dtype=torch.int32)
    broken[..., :13] = idx
    c = int(count[1, 2, 0])
    broken[1, 2, 0, :c + 2] = torch.cat((broken[1, 2, 0, :2], broken[1, 2, 0, 1:2], broken[1, 2, 0, 2:c],
                                        torch.tensor([40], device="cuda", dtype=torch.int32)))
    bc = count.clone()
    bc[1, 2, 0] = c + 2
    out, lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, block, broken, bc, 0.1, want_lse=True)
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() == 1                        # a repeat and one out of range, skipped
    check_tree(q, kc, vc, parents, block, keep, 0.1, None, out, lse)
    lens = torch.tensor([-3, T], device="cuda", dtype=torch.int32)
    out, lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, block, idx, count, 0.1, lens=lens, want_lse=True)
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() == 2                        # clamped to 0 and T - n
    check_tree(q, kc, vc, parents, block, keep, 0.1, torch.tensor([0, T - n]), out, lse)


def test_tree_of_one_node_is_decode():
    g = gen(10)
    q, kc, vc = randn(g, 2, 8, 1, 128), randn(g, 2, 2, 3000, 128), randn(g, 2, 2, 3000, 128)
    mean, var = spa.spa_block_stats(kc, 64)
    idx, count = spa.spa_select(q, mean, var, 3000, 64, 0.09, 0.8)
    a = spa.spa_sparse_attn_decode(q, kc, vc, 64, idx, count, 0.09)
    parents = torch.full((2, 1), -1, device="cuda", dtype=torch.int32)
    b, _ = spa.spa_sparse_attn_tree(q, kc, vc, parents, 64, idx, count, 0.09)
    # each rounds P and its result to bf16 (random weights: |out| well below 1)
    assert bool(((a.double() - b.double()).abs() <= 4 * U * (0.25 + a.double().abs())).all())
    r = spa.decode_tree(q, kc, vc, parents, 64, 0.8, scale=0.09, want_lse=True)
    assert torch.equal(r["out"], b) and torch.equal(r["idx"], idx) and r["lse"].shape == (2, 8, 1)
    ok()


def test_wrong_shapes_types_and_strides_are_refused():
    g = gen(16)
    q, kc, vc = randn(g, 1, 4, 3, 128), randn(g, 1, 2, 50, 128), randn(g, 1, 2, 50, 128)
    parents = torch.full((1, 3), -1, device="cuda", dtype=torch.int32)
    idx, count = torch.zeros(1, 4, 1, 4, device="cuda", dtype=torch.int32), torch.zeros(1, 4, 1, device="cuda", dtype=torch.int32)
    call = spa.spa_sparse_attn_tree
    for args in ((q, kc, vc[:, :1], parents, 16, None, None, 0.1), (q, kc, vc, parents.long(), 16, None, None, 0.1),
                 (q, kc, vc, parents[:, :2], 16, None, None, 0.1), (q.float(), kc, vc, parents, 16, None, None, 0.1),
                 (q, kc.transpose(1, 2).contiguous().transpose(1, 2), vc, parents, 16, None, None, 0.1),
                 (q, kc, vc, parents, 16, idx, None, 0.1), (q, kc, vc, parents, 16, idx, count[:, :2], 0.1)):
        with pytest.raises(ValueError):
            call(*args)
    with pytest.raises(spa.SpaError):
        call(q, kc, vc, parents, 16, None, None, 0.1, workspace=torch.empty(64, device="cuda", dtype=torch.uint8))
    freqs, _ = spa.spa_rope_frequencies(128)
    for bad in (freqs.float(), freqs.cuda(), freqs.reshape(2, 32)):
        with pytest.raises(ValueError):
            spa.spa_rope(q, None, bad)
    with pytest.raises(ValueError):
        spa.spa_rope(q.transpose(2, 3), None, freqs)                # features not contiguous
    with pytest.raises(ValueError):
        spa.spa_attn_weight(q, kc, torch.zeros(1, 4, 2, device="cuda"), 0.1)
    with pytest.raises(ValueError):
        spa.spa_cache_gather(kc, vc, idx.reshape(1, 4, 4))
    ok()


# ---------------------------------------------------------------- accumulated weight

def ref_weight(q, k, lse, scale, block, keep, lens, prev, decay):
    B, Hq, Lq, d = q.shape
    Hkv, T = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, Hkv, T, dtype=torch.float64, device="cuda")
    tol = out.clone()
    if prev is not None:
        out += prev.double() * decay
        tol += out.abs() * 2 * E
    for b in range(B):
        n = T if lens is None else int(lens[b])
        at = n - Lq + torch.arange(Lq, device="cuda")
        t = torch.arange(n, device="cuda")
        for h in range(Hq):
            K, x = k[b, h // G, :n].double(), q[b, h].double()
            s = (x @ K.T) * scale - lse[b, h].double()[:, None]
            see = (t[None] <= at[:, None]) & (lse[b, h] > -math.inf)[:, None]
            if keep is not None:
                see &= keep[b, h][at // block - (n - Lq) // block][:, t // block]
            w = torch.where(see, s.exp(), 0.0)
            out[b, h // G, :n] += w.sum(0)
            # the exponent's error: the logit's 2^-17 |q||k| (128 roundings), the log2
            # scaling's and the log-sum-exp's few E of its size; then the sum's roundings
            d_ = (x.abs() @ K.abs().T) * scale * 2.0 ** -17 + (8 * E * (s.abs() + lse[b, h].double().abs().nan_to_num(posinf=0)[:, None]) + 2.0 ** -21)
            tol[b, h // G, :n] += torch.where(see, w * (2 * d_ + (Lq * G + 4) * E), 0.0).sum(0)
    return out, tol


@pytest.mark.parametrize("B,Hq,Hkv,Lq,T,d,block,p,ragged", [
    (1, 1, 1, 1, 1, 128, 16, None, False),
    (3, 8, 2, 1, 1000, 128, 16, 0.5, True),
    (2, 16, 1, 1, 515, 64, 128, 0.5, False),
    (2, 10, 2, 33, 700, 128, 64, None, True),
    (1, 8, 2, 128, 128, 64, 32, None, False),          # all queries of a short prompt
    (1, 8, 2, 300, 1111, 128, 64, 0.5, False),         # a window over several query blocks
    (1, 3, 3, 257, 257, 128, 16, 0.3, False),
    (2, 4, 4, 2, 4097, 128, 32, None, True),
    (1, 16, 1, 200, 333, 128, 128, None, True),
    (1, 5, 1, 130, 260, 64, 128, 0.7, False),
    (40, 4, 2, 1, 300, 64, 16, None, True),            # more sequences than lanes
    (1, 8, 2, 1, 40001, 128, 16, 0.4, False),          # lists beyond a thousand entries
    (1, 4, 4, 4, 50, 128, 16, 0.6, False),             # four queries over two query blocks
    (1, 8, 2, 16, 3001, 128, 64, None, False),         # one query tile of 64 rows
    (1, 8, 2, 1500, 2500, 128, 128, None, False),      # runs of several pairs, joined
    (35, 8, 1, 40, 200, 64, 64, None, True),
])
def test_weight_matches_fp64(B, Hq, Hkv, Lq, T, d, block, p, ragged):
    g = gen(T + Lq)
    q, k = randn(g, B, Hq, Lq, d), randn(g, B, Hkv, T, d)
    lens = None
    if ragged:
        lens = torch.randint(Lq, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        lens[0] = Lq
        for b in range(B):
            k[b, :, int(lens[b]):] = float("nan")
    idx = count = keep = None
    if p is not None:
        nb, nq = -(-T // block), (T - 1) // block - (T - Lq) // block + 1
        keep = torch.rand(B, Hq, nq, nb, generator=g, device="cuda") < p
        j = torch.arange(nb, device="cuda", dtype=torch.int32)
        idx = torch.where(keep, j, nb + 3).sort(dim=3).values.to(torch.int32).contiguous()
        count = keep.sum(3).to(torch.int32)
        if ragged:
            keep = keep[:, :, :1]
    lse = torch.randn(B, Hq, Lq, generator=g, device="cuda") + math.log(T)
    lse[0, 0, Lq // 2] = -math.inf                      # a row that saw nothing
    prev = torch.rand(B, Hkv, T, generator=g, device="cuda")
    for pv, decay in ((None, 1.0), (prev, 0.75)):
        got = spa.spa_attn_weight(q, k, lse, SCALE[d], block, idx, count, lens=lens, prev=pv, decay=decay)
        ok()
        want, tol = ref_weight(q, k, lse, SCALE[d], block, keep, lens, pv, decay)
        assert bool(((got.double() - want).abs() <= tol).all()), float(((got.double() - want).abs() / tol.clamp(min=1e-30)).max())
    into = prev.clone()
    spa.spa_attn_weight(q, k, lse, SCALE[d], block, idx, count, lens=lens, prev=into, decay=0.75, out=into)
    assert torch.equal(into, got)                       # in place, and the same bits again


@pytest.mark.parametrize("B,Hq,Hkv,Lq,T,d,block,p,ragged", [
    (1, 4, 2, 100, 102301, 128, 128, None, False),     # ten key tiles per CTA, of one pair each
    (2, 8, 2, 300, 20003, 128, 64, None, True),        # five query tiles, some twenty pairs per CTA
    (2, 8, 2, 300, 6001, 64, 128, 0.5, False),
    (1, 8, 2, 16, 100001, 64, 32, None, False),        # a tile of 64 rows, ten key tiles per CTA
])
def test_weight_of_long_runs_matches_fp64(B, Hq, Hkv, Lq, T, d, block, p, ragged):
    test_weight_matches_fp64(B, Hq, Hkv, Lq, T, d, block, p, ragged)


def test_weight_lists_and_lengths_out_of_range_are_recorded():
    g = gen(11)
    q, k = randn(g, 1, 2, 1, 128), randn(g, 1, 1, 300, 128)
    lse = torch.full((1, 2, 1), 6.0, device="cuda")
    idx = torch.tensor([0, 3, 3, 2, 50], device="cuda", dtype=torch.int32).expand(1, 2, 1, 5).contiguous()
    count = torch.full((1, 2, 1), 5, device="cuda", dtype=torch.int32)
    got = spa.spa_attn_weight(q, k, lse, 0.09, 64, idx, count)
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() == 1
    keep = torch.zeros(1, 2, 1, 5, dtype=torch.bool, device="cuda")
    keep[..., [0, 3]] = True
    want, tol = ref_weight(q, k, lse, 0.09, 64, keep, None, None, 1.0)
    assert bool(((got.double() - want).abs() <= tol).all())
    lens = torch.tensor([301], device="cuda", dtype=torch.int32)
    got = spa.spa_attn_weight(q, k, lse, 0.09, lens=lens)
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() == 2
    want, tol = ref_weight(q, k, lse, 0.09, 64, None, None, None, 1.0)
    assert bool(((got.double() - want).abs() <= tol).all())


def test_weight_of_attention_sums_to_its_queries():
    # with attention's own log-sum-exp every query hands out a weight of 1 in all
    g = gen(12)
    q, k, v = randn(g, 1, 8, 640, 128), randn(g, 1, 2, 640, 128), randn(g, 1, 2, 640, 128)
    r = spa.prefill(q, k, v, 128, 0.7, want_lse=True)
    w = spa.spa_attn_weight(q, k, r["lse"], 128.0 ** -0.5, 128, r["idx"], r["count"])
    ok()
    assert abs(float(w.double().sum()) / (8 * 640) - 1) < 1e-4


# ---------------------------------------------------------------- eviction

def ref_evict(score, lens, n_keep, n_sink, n_recent):
    B, Hkv, T = score.shape
    keep = torch.full((B, Hkv, n_keep), -1, dtype=torch.int32)
    count = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        n = T if lens is None else int(lens[b])
        count[b] = c = min(n, n_keep)
        for g in range(Hkv):
            s = score[b, g, :n].tolist()
            fixed = lambda t: t < n_sink or t >= n - n_recent   # noqa: E731
            low = lambda x: -math.inf if x != x else x          # noqa: E731
            best = sorted(range(n), key=lambda t: (not fixed(t), s[t] != s[t], -low(s[t]), t))[:c]
            keep[b, g, :c] = torch.tensor(sorted(best), dtype=torch.int32)
    return keep, count


@pytest.mark.parametrize("B,Hkv,T,n_keep,n_sink,n_recent,ragged,kind", [
    (1, 1, 1, 1, 0, 0, False, "random"), (1, 1, 5, 9, 2, 3, False, "random"), (2, 3, 100, 10, 4, 6, False, "random"),
    (2, 2, 1000, 333, 0, 0, True, "random"), (3, 2, 1000, 999, 5, 100, True, "equal"), (1, 2, 4097, 1, 0, 0, False, "equal"),
    (1, 1, 40000, 5000, 4, 128, False, "few"), (2, 1, 20000, 19999, 1, 1, True, "random"),
    (1, 1, 400001, 3000, 4, 32, False, "random"),       # more keys than a cluster holds
    (1, 2, 70001, 512, 0, 64, False, "wild"), (2, 1, 9000, 4000, 8, 8, False, "wild"), (4, 1, 300, 64, 64, 0, True, "few"),
])
def test_evict_select_is_exact(B, Hkv, T, n_keep, n_sink, n_recent, ragged, kind):
    g = gen(T)
    score = torch.rand(B, Hkv, T, generator=g, device="cuda")
    if kind == "equal":
        score.fill_(0.25)
    if kind == "few":
        score = (score * 4).floor()
    if kind == "wild":
        score = (score - 0.5) * 1e30
        pick = torch.randint(0, T, (6, T // 10), generator=g, device="cuda")
        for at, x in zip(pick, (math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42)):
            score[..., at] = x
    lens = None
    if ragged:
        lens = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        lens[0] = 0
        score[0] = math.nan
    keep, count = spa.spa_evict_select(score, n_keep, n_sink, n_recent, lens=lens)
    ok()
    wk, wc = ref_evict(score, lens, n_keep, n_sink, n_recent)
    assert torch.equal(count.cpu(), wc) and torch.equal(keep.cpu(), wk)


def test_evict_lengths_out_of_range_are_recorded():
    score = torch.rand(2, 1, 50, generator=gen(1), device="cuda")
    lens = torch.tensor([-1, 51], device="cuda", dtype=torch.int32)
    keep, count = spa.spa_evict_select(score, 7, lens=lens)
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() == 2 and count.tolist() == [0, 7]
    assert torch.equal(keep.cpu(), ref_evict(score, [0, 50], 7, 4, 0)[0])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64), (BF, 8), (F32, 256)])
def test_cache_gather_moves_rows_and_leaves_the_rest(dtype, d):
    g = gen(d)
    B, Hkv, T, n_keep, T_out = 3, 2, 200, 37, 40
    kc, vc = randn(g, B, Hkv, T, d, dtype=dtype), randn(g, B, Hkv, T, d, dtype=dtype)
    score = torch.rand(B, Hkv, T, generator=g, device="cuda")
    keep = torch.randint(0, T, (B, Hkv, n_keep), generator=g, device="cuda", dtype=torch.int32)
    count = torch.tensor([37, 0, 12], device="cuda", dtype=torch.int32)
    ko, vo = (torch.full((B, Hkv, T_out, d), 9.0, device="cuda", dtype=dtype) for _ in range(2))
    so = torch.full((B, Hkv, T_out), 9.0, device="cuda")
    wk, wv, ws = ko.clone(), vo.clone(), so.clone()
    spa.spa_cache_gather(kc, vc, keep, count, score=score, k_out=ko, v_out=vo, score_out=so)
    ok()
    for b, c in enumerate(count.tolist()):
        for h in range(Hkv):
            t = keep[b, h, :c].long()
            wk[b, h, :c], wv[b, h, :c], ws[b, h, :c] = kc[b, h, t], vc[b, h, t], score[b, h, t]
    assert torch.equal(ko, wk) and torch.equal(vo, wv) and torch.equal(so, ws)
    k1, v1, s1 = spa.spa_cache_gather(kc, vc, keep)                 # every entry of the list
    at = keep.long()[..., None].expand(-1, -1, -1, d)
    assert s1 is None and torch.equal(k1, kc.gather(2, at)) and torch.equal(v1, vc.gather(2, at))
    keep[0, 1, 3], keep[0, 0, 5] = -1, T
    spa.spa_cache_gather(kc, vc, keep, torch.tensor([37, 38, -1], device="cuda", dtype=torch.int32), k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    assert spa.spa_get_device_error() in (1, 2)
    t = keep[1, 0].long()
    wk[1, 0, :n_keep] = kc[1, 0, t]
    t = keep[1, 1].long()
    wk[1, 1, :n_keep] = kc[1, 1, t]
    assert torch.equal(ko, wk)                       # the bad entries and the negative count: as they were


# ---------------------------------------------------------------- together

def serve_once(s, stream=None):
    """A step of drafted tokens on a long cache, then an eviction; torch's copies between
    the calls are made on the calls' stream."""
    r = {}

    def dense(x):
        with torch.cuda.stream(stream):               # None: the current one
            return x.contiguous()

    r["q"] = spa.spa_rope_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], *s["rope"], row0=s["len"], pos=s["pos"],
                                 stream=stream)
    mean, var = spa.spa_block_stats(s["kc"], 32, stream=stream)
    root = dense(r["q"][:, :, :1])
    idx, count = spa.spa_select(root, mean, var, s["kc"].shape[2], 32, s["scale"], 0.8, stream=stream)
    r["out"], r["lse"] = spa.spa_sparse_attn_tree(r["q"], s["kc"], s["vc"], s["parents"], 32, idx, count, s["scale"],
                                                  want_lse=True, stream=stream)
    # the newest token's weight on the keys it attended to
    last = dense(r["q"][:, :, -1:])
    r["w"] = spa.spa_attn_weight(last, s["kc"], dense(r["lse"][:, :, -1:]), s["scale"], 32, idx, count,
                                 prev=s["w"], stream=stream)
    e = spa.evict(s["kc"], s["vc"], r["w"], 500, 4, 64, stream=stream)
    r.update(keep=e["keep"], k2=e["k"], v2=e["v"], w2=e["score"], idx=idx, count=count)
    m2, v2 = spa.spa_block_stats(e["k"], 32, stream=stream)
    i2, c2 = spa.spa_select(root, m2, v2, 500, 32, s["scale"], 0.9, stream=stream)
    r["dec"] = spa.spa_sparse_attn_decode(root, e["k"], e["v"], 32, i2, c2, s["scale"], stream=stream)
    return r


def serving_state(seed):
    g = gen(seed)
    B, Hq, Hkv, n, T, d = 2, 8, 2, 6, 1500, 128
    qkv = randn(g, B, n, Hq + 2 * Hkv, d).transpose(1, 2)
    parents = torch.tensor([[-1, 0, 0, 1, 2, 4]] * B, device="cuda", dtype=torch.int32)
    depth = torch.tensor([[0, 1, 1, 2, 2, 3]] * B, device="cuda", dtype=torch.int32)
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], kc=randn(g, B, Hkv, T, d),
                vc=randn(g, B, Hkv, T, d), rope=spa.spa_rope_frequencies(d), len=T - n, pos=depth + T - n,
                parents=parents, scale=d ** -0.5, w=torch.rand(B, Hkv, T, generator=g, device="cuda"))


def test_a_step_and_an_eviction_together():
    s = serving_state(20)
    r = serve_once(s)
    ok()
    T, n = s["kc"].shape[2], 6
    want, mag = ref_rope(s["k"], s["pos"], s["rope"][0], 1.0, "half")
    close_rope(s["kc"][:, :, T - n:], want, mag, BF)
    nb = -(-T // 32)
    keep = torch.zeros(2, 8, 1, nb + 1, dtype=torch.bool, device="cuda")
    at = torch.arange(r["idx"].shape[3], device="cuda") < r["count"][..., None]
    keep.scatter_(3, torch.where(at, r["idx"], nb).long(), at)
    check_tree(r["q"], s["kc"], s["vc"], s["parents"], 32, keep[..., :nb], s["scale"], None, r["out"], r["lse"])
    wk, _ = ref_evict(r["w"], None, 500, 4, 64)
    assert torch.equal(r["keep"].cpu(), wk)
    t = wk.long().cuda()
    assert torch.equal(r["k2"], s["kc"].gather(2, t[..., None].expand(-1, -1, -1, 128)))
    assert torch.equal(r["w2"], r["w"].gather(2, t)) and bool(torch.isfinite(r["dec"].float()).all())


def test_the_same_step_on_another_stream_and_replayed_from_a_graph():
    a, b = serving_state(21), serving_state(22)
    want = [serve_once(a), serve_once(b)]
    want = [{k: v.clone() for k, v in w.items()} for w in want]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = serve_once(a, stream=side)
    torch.cuda.synchronize()
    for k in want[0]:
        if k not in ("idx",):
            assert torch.equal(got[k], want[0][k]), k
    graphs, outs = [], []
    for s in (a, b):                                  # two graphs, replayed in turn and again
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(serve_once(s))
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for k in w:
            if k not in ("idx",):
                assert torch.equal(o[k], w[k]), k
    ok()


def test_prefill_takes_unrotated_inputs():
    g = gen(23)
    qkv = randn(g, 1, 300, 8 + 2, 128).transpose(1, 2)
    v = randn(g, 1, 2, 300, 128)
    rope = spa.spa_rope_frequencies(128)
    r = spa.prefill(qkv[:, :8], qkv[:, 8:], v, 128, 0.9, rope=rope)
    q, k = spa.spa_rope(qkv[:, :8], qkv[:, 8:], *rope)
    w = spa.prefill(q, k, v, 128, 0.9)
    assert torch.equal(r["out"], w["out"]) and torch.equal(r["k"], k) and torch.equal(r["q"], q)
    ok()
