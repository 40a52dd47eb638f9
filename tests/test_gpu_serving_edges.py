"""The serving operators at the edges of what their documentation allows: values that are
not finite, tensors that start anywhere, drafted rows, trees with branches. Helpers and
tolerances are those of test_gpu_serving."""
import math

import pytest
import torch

import block_sparse_long_stats_b200 as spa
from tests.test_gpu_serving import (BF, E, SCALE, U, check_tree, gen, lists, ok, randn, ref_tree, ref_weight,
                                    tree_of)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- values that are not finite

# one tile per run, so that every unit is joined; and units that one run finishes
@pytest.mark.parametrize("B,Hq,Hkv,n,T", [(1, 4, 2, 5, 700), (80, 8, 4, 3, 140), (1, 10, 1, 33, 1300)])
@pytest.mark.parametrize("where", ["query", "text key", "drafted key", "infinite key", "text value"])
def test_tree_gives_what_the_definition_does_for_values_that_are_not_finite(B, Hq, Hkv, n, T, where):
    g = gen(T + n)
    q, kc, vc = randn(g, B, Hq, n, 128), randn(g, B, Hkv, T, 128), randn(g, B, Hkv, T, 128)
    parents = tree_of(g, B, n)
    parents[:, -1] = -2                               # an unused node: never touched
    clean, clean_lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, 64, None, None, 0.09, want_lse=True)
    P, hit = T - n, torch.zeros(B, Hq, n, dtype=torch.bool, device="cuda")
    G = Hq // Hkv
    if where == "query":
        q[0, 1, 1, 7] = math.nan
        hit[0, 1, 1] = True
    elif where == "text key":
        kc[-1, 0, P // 2, 3] = math.nan
        hit[-1, :G] = True
    elif where == "drafted key":                      # node 0: its descendants see it
        kc[-1, -1, P, 3] = math.nan
        for i in range(n):
            j = i
            while j > 0:
                j = int(parents[-1, j])
            hit[-1, -G:, i] = j == 0
    elif where == "infinite key":                     # +inf and -inf scores, by the query's sign
        kc[0, 0, 0, 11] = math.inf
        q[0, :G, 0, 11], q[0, :G, 1, 11] = 2.0, -2.0
        q[0, :G, :, 11] += (q[0, :G, :, 11] == 0).to(BF)
        hit[0, :G] = q[0, :G, :, 11] > 0
    else:
        vc[0, 0, 0, 5] = math.inf
    hit &= (parents >= -1)[:, None]
    out, lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, 64, None, None, 0.09, want_lse=True)
    ok()
    if where == "text value":                         # lse without a trace, one feature infinite
        assert torch.equal(lse, clean_lse)
        live = (parents[0] >= -1).expand(G, n)
        assert bool((out[0, :G, :, 5][live] == math.inf).all())
        out[0, :G, :, 5] = clean[0, :G, :, 5]
        assert torch.equal(out, clean)
        return
    assert bool(hit.any()) and bool(torch.isnan(lse[hit]).all()) and bool(torch.isnan(out[hit]).all())
    rest = ~hit
    if where == "infinite key":                       # a score of -inf: a key without weight
        assert bool(torch.isfinite(out[rest].float()).all())
        want, wl, mag, qk = ref_tree(q[:1, :G], kc[:1, :1, 1:], vc[:1, :1, 1:], parents[:1], 64, None, 0.09, None)
        d, r = 2.0 ** -17 * qk + 2.0 ** -18, (rest & (parents >= -1)[:, None])[:1, :G]
        tol = (1.02 * U + 2 * d[..., None]) * mag + U * want.abs()
        assert bool(r.any()) and bool(((out[:1, :G].double() - want).abs() <= tol)[r].all())
    else:
        assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])


# one query tile per head in registers, 64 and 128 columns, and streams of query tiles
@pytest.mark.parametrize("Hq,Hkv,Lq,T,d,block,p", [
    (8, 2, 1, 1000, 128, 16, None), (8, 2, 4, 515, 64, 32, 0.6), (8, 2, 13, 700, 128, 64, None),
    (8, 2, 31, 900, 64, 64, 0.5), (5, 1, 25, 400, 128, 128, None), (8, 2, 130, 1111, 128, 64, None),
    (10, 2, 130, 1111, 64, 128, 0.5), (4, 4, 700, 700, 128, 128, None)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_query_that_saw_nothing_adds_nothing_whatever_it_holds(Hq, Hkv, Lq, T, d, block, p, bad):
    g = gen(T + Lq + Hq)
    q, k = randn(g, 2, Hq, Lq, d), randn(g, 2, Hkv, T, d)
    idx = count = None
    if p is not None:
        nb, nq = -(-T // block), (T - 1) // block - (T - Lq) // block + 1
        keep = torch.rand(2, Hq, nq, nb, generator=g, device="cuda") < p
        j = torch.arange(nb, device="cuda", dtype=torch.int32)
        idx = torch.where(keep, j, nb).sort(dim=3).values.to(torch.int32).contiguous()
        count = keep.sum(3).to(torch.int32)
    lse = torch.randn(2, Hq, Lq, generator=g, device="cuda") + math.log(T)
    dead = torch.rand(2, Hq, Lq, generator=g, device="cuda") < 0.3
    dead[0, 0, 0] = dead[1, -1, -1] = True
    lse[dead] = -math.inf
    q[dead] = 0.0
    want = spa.spa_attn_weight(q, k, lse, SCALE[d], block, idx, count)
    q[dead] = bad
    q[0, 0, 0, 1:] = 0.0                              # one feature is enough
    got = spa.spa_attn_weight(q, k, lse, SCALE[d], block, idx, count)
    ok()
    assert bool(torch.isfinite(want).all()) and torch.equal(got, want)
    lse[0, 0, 0] = 1.0                                # a query that saw keys is not hidden
    got = spa.spa_attn_weight(q, k, lse, SCALE[d], block, idx, count)
    if p is None and math.isnan(bad):
        assert bool(torch.isnan(got[0, 0, 0]))
    assert torch.equal(got[1], want[1])
    ok()


@pytest.mark.parametrize("T", [17, 33, 4095, 4097, 4111])
@pytest.mark.parametrize("Lq,d", [(1, 128), (2, 64)])
def test_weight_of_a_cache_that_ends_inside_a_slab(T, Lq, d):
    # the last slab of 16 keys is cut by the end of the tensor
    g = gen(T + d)
    q, k = randn(g, 2, 4, Lq, d), randn(g, 2, 2, T, d)
    lse = torch.randn(2, 4, Lq, generator=g, device="cuda") + math.log(T)
    got = spa.spa_attn_weight(q, k, lse, SCALE[d])
    ok()
    want, tol = ref_weight(q, k, lse, SCALE[d], 128, None, None, None, 1.0)
    assert bool(((got.double() - want).abs() <= tol).all())


# ---------------------------------------------------------------- drafted rows

@pytest.mark.parametrize("n,T,block", [(64, 1024, 16), (64, 1030, 16), (33, 1500, 32), (2, 1001, 16), (128, 700, 64)])
def test_decode_tree_selects_from_the_committed_text(n, T, block):
    g = gen(T + n)
    B, Hq, Hkv, P = 2, 8, 2, T - n
    q, kc, vc = randn(g, B, Hq, n, 128), randn(g, B, Hkv, T, 128), randn(g, B, Hkv, T, 128)
    parents = tree_of(g, B, n)
    r = spa.decode_tree(q, kc, vc, parents, block, 0.6, want_lse=True)
    ok()
    nb, kept = -(-P // block), torch.zeros(B, Hq, 1, -(-T // block) + 1, dtype=torch.bool, device="cuda")
    assert r["idx"].shape[3] >= -(-T // block)
    at = torch.arange(r["idx"].shape[3], device="cuda") < r["count"][..., None]
    kept.scatter_(3, torch.where(at, r["idx"], kept.shape[3] - 1).long(), at)
    kept = kept[..., :-1]
    assert bool(kept[..., nb - 1].all()) and bool(kept[..., 0].all()) and not bool(kept[..., nb:].any())
    # the lists of the text alone, its newest row as the position
    m, v = spa.spa_block_stats(kc[:, :, :P].contiguous(), block)
    i, c = spa.spa_select(q[:, :, :1].contiguous(), m, v, P, block, 128.0 ** -0.5, 0.6)
    assert torch.equal(c, r["count"]) and torch.equal(i[at[..., :nb]], r["idx"][at])
    assert torch.equal(m, r["mean"]) and torch.equal(v, r["var"])
    check_tree(q, kc, vc, parents, block, kept, 128.0 ** -0.5, None, r["out"], r["lse"])
    # whatever the drafted rows hold; with the statistics given, of the text or of more blocks
    kc[:, :, P:] = 30.0
    more = [torch.cat((x, torch.full((B, Hkv, 3, 128), math.nan, device="cuda")), 2) for x in (m, v)]
    for kw in ({}, dict(mean=m, var=v), dict(mean=more[0], var=more[1])):
        s = spa.decode_tree(q, kc, vc, parents, block, 0.6, **kw)
        assert torch.equal(s["count"], r["count"]) and torch.equal(s["idx"][at], r["idx"][at])
    ok()


def test_decode_tree_without_text_and_of_one_node():
    g = gen(31)
    q, kc, vc = randn(g, 2, 8, 20, 128), randn(g, 2, 2, 20, 128), randn(g, 2, 2, 20, 128)
    parents = tree_of(g, 2, 20)
    r = spa.decode_tree(q, kc, vc, parents, 16, 0.6, want_lse=True)
    ok()
    assert int(r["count"].sum()) == 0
    check_tree(q, kc, vc, parents, 16, None, 128.0 ** -0.5, None, r["out"], r["lse"])
    for T in (1000, 1025):                            # the tree of one node is a decode step
        q, kc, vc = randn(g, 2, 8, 1, 128), randn(g, 2, 2, T, 128), randn(g, 2, 2, T, 128)
        one = torch.full((2, 1), -1, device="cuda", dtype=torch.int32)
        a, b = spa.decode_tree(q, kc, vc, one, 32, 0.6), spa.decode(q, kc, vc, 32, 0.6)
        at = torch.arange(a["idx"].shape[3], device="cuda") < a["count"][..., None]
        assert torch.equal(a["count"], b["count"]) and torch.equal(a["idx"][at], b["idx"][at])
    ok()


# ---------------------------------------------------------------- from a tree to the accumulated weight

def check_shares(q, kc, lse, scale, block, keep, lens, w):
    """w is the queries' weight on the keys they attended to: key by key, and one in all for
    each query and head."""
    want, tol = ref_weight(q, kc, lse, scale, block, keep, lens, None, 1.0)
    assert bool(((w.double() - want).abs() <= tol).all())
    # the log-sum-exp's own error: 2^-17 of |q||k| summed over the features and 2^-18, 4 E of its size
    G, Lq = q.shape[1] // kc.shape[1], q.shape[2]
    k = kc.double().abs().nan_to_num().repeat_interleave(G, 1)
    d = 2.0 ** -17 * scale * (q.double().abs() @ k.transpose(2, 3)).amax(3) + 2.0 ** -18 + 4 * E * lse.double().abs()
    slack = tol.sum(2) + 2 * d.reshape(*w.shape[:2], -1).sum(2)
    assert bool(((w.double().sum(2) - G * Lq).abs() <= slack).all())


@pytest.mark.parametrize("n,block", [(1, 32), (9, 16), (40, 16), (40, 64)])
def test_weight_of_a_chain_over_lists_sums_to_its_queries(n, block):
    # drafts in a line; the lists get the blocks that the drafts lie in
    g = gen(n + block)
    B, Hq, Hkv, T = 2, 8, 2, 1003
    P, nb = T - n, -(-T // block)
    q, kc, vc = randn(g, B, Hq, n, 128), randn(g, B, Hkv, T, 128), randn(g, B, Hkv, T, 128)
    parents = (torch.arange(n, device="cuda", dtype=torch.int32) - 1).expand(B, n).contiguous()
    r = spa.decode_tree(q, kc, vc, parents, block, 0.5, want_lse=True)
    j = torch.arange(nb, device="cuda")
    keep = torch.zeros(B, Hq, 1, nb + 1, dtype=torch.bool, device="cuda")
    at = torch.arange(r["idx"].shape[3], device="cuda") < r["count"][..., None]
    keep = keep.scatter_(3, torch.where(at, r["idx"], nb).long(), at)[..., :nb] | (j >= P // block)
    nq = (T - 1) // block - P // block + 1
    keep = keep.expand(B, Hq, nq, nb)
    idx = torch.where(keep, j, nb).sort(dim=3).values.to(torch.int32).contiguous()
    w = spa.spa_attn_weight(q, kc, r["lse"], 128.0 ** -0.5, block, idx, keep.sum(3).to(torch.int32))
    ok()
    check_shares(q, kc, r["lse"], 128.0 ** -0.5, block, keep, None, w)


def test_weight_of_an_accepted_path_and_of_the_root_sums_to_its_queries():
    # a tree with branches in ragged caches: the root as it is, the path once its rows follow
    # one another
    g = gen(61)
    B, Hq, Hkv, T, n, scale = 3, 8, 2, 600, 7, 128.0 ** -0.5
    q, kc, vc = randn(g, B, Hq, n, 128), randn(g, B, Hkv, T, 128), randn(g, B, Hkv, T, 128)
    parents = torch.tensor([[-1, 0, 0, 1, 2, 4, 2]] * B, device="cuda", dtype=torch.int32)
    lens = torch.tensor([0, 77, T - n], device="cuda", dtype=torch.int32)
    out, lse = spa.spa_sparse_attn_tree(q, kc, vc, parents, 64, None, None, scale, lens=lens, want_lse=True)
    q1, lse1 = q[:, :, :1].contiguous(), lse[:, :, :1].contiguous()
    check_shares(q1, kc, lse1, scale, 64, None, lens + 1, spa.spa_attn_weight(q1, kc, lse1, scale, lens=lens + 1))
    path = torch.tensor([0, 2, 4, 5], device="cuda")
    b = torch.arange(B, device="cuda")[:, None]
    for c in (kc, vc):
        c[b, :, lens[:, None] + torch.arange(4, device="cuda")] = c[b, :, lens[:, None] + path]
    qp, lp = q[:, :, path].contiguous(), lse[:, :, path].contiguous()
    w = spa.spa_attn_weight(qp, kc, lp, scale, lens=lens + 4)
    ok()
    check_shares(qp, kc, lp, scale, 64, None, lens + 4, w)


# ---------------------------------------------------------------- tensors that start anywhere

def test_weight_takes_fp32_tensors_that_start_at_any_element():
    g = gen(41)
    for Lq, T in ((1, 515), (33, 301), (200, 777)):
        q, k = randn(g, 3, 3, Lq, 128), randn(g, 3, 1, T, 128)
        lse = torch.randn(3, 3, Lq, generator=g, device="cuda") + math.log(T)
        prev = torch.rand(3, 1, T, generator=g, device="cuda")
        want = spa.spa_attn_weight(q, k, lse, 0.09, prev=prev, decay=0.5)
        out = torch.full_like(prev, 7.0)
        for b in range(3):                            # batch slices: 4-byte aligned
            spa.spa_attn_weight(q[b:b + 1].contiguous(), k[b:b + 1].contiguous(), lse[b:b + 1], 0.09,
                                prev=prev[b:b + 1], decay=0.5, out=out[b:b + 1])
        ok()
        for b in range(3):
            ww, tol = ref_weight(q[b:b + 1], k[b:b + 1], lse[b:b + 1], 0.09, 128, None, None, prev[b:b + 1], 0.5)
            assert bool(((out[b:b + 1].double() - ww).abs() <= tol).all())
            assert bool(((want[b:b + 1].double() - ww).abs() <= tol).all())


def test_new_outputs_of_the_gather_are_zero_behind_the_list():
    # k_out is given with more rows than the list; the new v_out and score_out have as many
    g = gen(71)
    kc, vc = randn(g, 2, 2, 60, 128), randn(g, 2, 2, 60, 128)
    score = torch.rand(2, 2, 60, generator=g, device="cuda")
    keep = torch.randint(0, 60, (2, 2, 7), generator=g, device="cuda", dtype=torch.int32)
    for _ in range(3):                                # memory that held something else
        junk = [torch.full((2, 2, 500, 128), 3.0, device="cuda", dtype=BF), torch.full((2, 2, 500), 3.0, device="cuda")]
        del junk
        k_out = torch.full((2, 2, 500, 128), 5.0, device="cuda", dtype=BF)
        k, v, s = spa.spa_cache_gather(kc, vc, keep, score=score, k_out=k_out)
        ok()
        assert k is k_out and v.shape == k.shape and s.shape == (2, 2, 500)
        assert bool((k[:, :, 7:] == 5).all() and (v[:, :, 7:] == 0).all() and (s[:, :, 7:] == 0).all())
        at = keep.long()
        assert torch.equal(v[:, :, :7], vc.gather(2, at[..., None].expand(2, 2, 7, 128)))
        assert torch.equal(s[:, :, :7], score.gather(2, at))


# ---------------------------------------------------------------- captured, on another stream

@pytest.mark.parametrize("d,n,T,block", [(64, 20, 500, 32), (128, 9, 1200, 64), (128, 60, 70, 16)])
def test_decode_tree_on_another_stream_and_replayed_from_a_graph(d, n, T, block):
    # the last one: less text than a block
    g = gen(81 + T)
    q, kc, vc = randn(g, 2, 8, n, d), randn(g, 2, 2, T, d), randn(g, 2, 2, T, d)
    parents = tree_of(g, 2, n)

    def same(r):
        at = torch.arange(want["idx"].shape[3], device="cuda") < want["count"][..., None]
        assert torch.equal(r["idx"][at], want["idx"][at])
        assert all(torch.equal(r[k], want[k]) for k in ("out", "lse", "count", "mean", "var"))

    want = {k: v.clone() for k, v in spa.decode_tree(q, kc, vc, parents, block, 0.6, want_lse=True).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = spa.decode_tree(q, kc, vc, parents, block, 0.6, want_lse=True, stream=side)
    torch.cuda.synchronize()
    same(r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = spa.decode_tree(q, kc, vc, parents, block, 0.6, want_lse=True)
    for _ in range(2):
        r["out"].zero_()
        graph.replay()
    torch.cuda.synchronize()
    same(r)
    ok()
