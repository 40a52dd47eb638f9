"""Refusals and host-side arithmetic of the serving operators (rotary positions, tree
attention, accumulated attention weight, eviction). CPU only: every refused call fails
a host check before any launch."""
import ctypes
import math

import pytest
import torch

import block_sparse_long_stats_b200 as spa
from block_sparse_long_stats_b200 import build as spa_build

P = ctypes.c_void_p
FAKE = 0x10000          # aligned, never dereferenced
OTHER = 0x20000
I, F, D, Z = ctypes.c_int, ctypes.c_float, ctypes.c_double, ctypes.c_size_t


@pytest.fixture(scope="module")
def lib():
    spa_build.build()
    return spa.lib()


def freqs(n):
    return (ctypes.c_double * n)(*[1.0] * n)


def test_rope_frequencies_follow_their_definitions(lib):
    f, m = spa.spa_rope_frequencies(64, 10000.0)
    want = torch.tensor([10000.0 ** (-2.0 * c / 64) for c in range(32)], dtype=torch.float64)
    assert m == 1.0 and torch.allclose(f, want, rtol=1e-14, atol=0)
    lin, m = spa.spa_rope_frequencies(64, 10000.0, "linear", factor=4.0)
    assert m == 1.0 and torch.allclose(lin, want / 4, rtol=1e-14, atol=0)
    ntk, _ = spa.spa_rope_frequencies(64, 10000.0, "ntk", factor=4.0)
    assert ntk[0] == 1.0 and abs(float(ntk[-1] / (want[-1] / 4)) - 1) < 1e-12   # slowest interpolated
    parts, m = spa.spa_rope_frequencies(64, 10000.0, "parts", factor=4.0, trained=4096)
    assert abs(m - (1 + 0.1 * math.log(4.0))) < 1e-7
    turns = 4096 * want / (2 * math.pi)
    ratio = parts / want
    assert torch.all(ratio[turns > 33] == 1.0) and torch.allclose(ratio[turns < 0.7], torch.tensor(0.25).double())
    assert torch.all(ratio[1:] <= ratio[:-1])                                    # a ramp between
    assert torch.all((ratio <= 1.0) & (ratio >= 0.25))


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(rot=258), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=2.0, rot=2),
                                dict(scaling="parts", factor=2.0, trained=0.0),
                                dict(scaling="parts", factor=2.0, trained=4096, fast=1.0, slow=1.0)])
def test_rope_frequencies_refusals(lib, kw):
    with pytest.raises(spa.SpaError) as e:
        spa.spa_rope_frequencies(**dict(dict(rot=64), **kw))
    assert e.value.status == 1


def test_unknown_names_are_refused(lib):
    with pytest.raises(ValueError):
        spa.spa_rope_frequencies(64, scaling="cubic")


def rope(lib, **kw):
    a = dict(q=FAKE, qo=OTHER, k=FAKE, ko=OTHER, dt=1, B=1, Hq=4, Hkv=2, L=8, d=128, rot=128, layout=0,
             f=freqs(64), m=1.0, pos0=0, backward=0)
    a.update(kw)
    return lib.spa_rope(a["q"], None, a["qo"], None, a["k"], None, a["ko"], None, a["dt"], a["B"], a["Hq"], a["Hkv"],
                        a["L"], a["d"], a["rot"], a["layout"], a["f"], a["m"], None, a["pos0"], a["backward"], None)


def test_rope_refusals(lib):
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(f=None), dict(B=0), dict(L=0), dict(Hkv=0), dict(dt=2),
               dict(layout=2), dict(rot=0), dict(rot=7), dict(rot=130), dict(m=float("inf")), dict(backward=2),
               dict(q=FAKE + 1), dict(pos0=0x7fffffff), dict(f=(ctypes.c_double * 64)(*[float("nan")] * 64))):
        assert rope(lib, **kw) == 1, kw
    assert rope(lib, d=512, rot=128) == 2
    assert rope(lib, B=1 << 16, L=1 << 16) == 2


def append(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, kc=OTHER, vc=OTHER, L=4, T=100, rows=None, row0=0, d=128, rot=64)
    a.update(kw)
    return lib.spa_rope_append(a["q"], None, OTHER, None, a["k"], None, a["v"], None, a["kc"], a["vc"], 1, 1, 4, 2,
                               a["L"], a["T"], a["d"], a["rot"], 0, freqs(64), 1.0, None, a["rows"], a["row0"], None)


def test_rope_append_refusals(lib):
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(T=0), dict(row0=-1),
               dict(row0=97), dict(rot=1), dict(L=101)):
        assert append(lib, **kw) == 1, kw
    assert append(lib, d=512) == 2


def tree(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, dt=1, B=1, Hq=8, Hkv=2, n=8, T=256, d=128, block=16, parents=FAKE, idx=FAKE,
             cap=16, count=FAKE, scale=0.1, ws=FAKE, out=FAKE)
    a.update(kw)
    need = lib.spa_tree_workspace_bytes(a["B"], a["Hq"], a["Hkv"], a["n"], a["T"], a["d"], a["block"])
    return lib.spa_sparse_attn_tree(a["q"], a["kc"], a["vc"], a["dt"], a["B"], a["Hq"], a["Hkv"], a["n"], a["T"],
                                    a["d"], a["block"], a["parents"], None, a["idx"], a["cap"], a["count"], a["scale"],
                                    a["ws"], a.get("nws", need), a["out"], None, None)


def test_tree_refusals(lib):
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(parents=None), dict(ws=None), dict(out=None),
               dict(idx=None), dict(count=None), dict(B=0), dict(n=0), dict(Hq=3), dict(n=9, T=8, cap=16),
               dict(scale=0.0), dict(scale=float("nan")), dict(cap=15), dict(q=FAKE + 8), dict(nws=0)):
        assert tree(lib, **kw) == 1, kw
    for kw in (dict(dt=0), dict(d=96), dict(block=48), dict(block=256), dict(n=129), dict(Hq=34),
               dict(B=64, T=1 << 26, cap=1 << 22)):
        assert tree(lib, **kw) == 2, kw
    assert lib.spa_tree_workspace_bytes(1, 8, 2, 129, 256, 128, 16) == 0
    assert lib.spa_tree_workspace_bytes(1, 8, 3, 8, 256, 128, 16) == 0
    assert lib.spa_tree_workspace_bytes(1, 8, 2, 8, 4, 128, 16) == 0


def weight(lib, **kw):
    a = dict(q=FAKE, k=FAKE, dt=1, B=1, Hq=8, Hkv=2, Lq=1, T=256, d=128, lse=FAKE, lens=None, block=16, idx=FAKE,
             cap=16, count=FAKE, scale=0.1, decay=1.0, ws=FAKE, out=FAKE)
    a.update(kw)
    need = lib.spa_attn_weight_workspace_bytes(a["B"], a["Hq"], a["Lq"], a["T"], a["block"])
    return lib.spa_attn_weight(a["q"], a["k"], a["dt"], a["B"], a["Hq"], a["Hkv"], a["Lq"], a["T"], a["d"], a["lse"],
                               a["lens"], a["block"], a["idx"], a["cap"], a["count"], a["scale"], None, a["decay"],
                               a["ws"], a.get("nws", need), a["out"], None)


def test_weight_refusals(lib):
    for kw in (dict(q=None), dict(k=None), dict(lse=None), dict(out=None), dict(idx=None), dict(count=None), dict(B=0),
               dict(Lq=0), dict(Lq=257), dict(Hq=3), dict(scale=-1.0), dict(decay=float("inf")), dict(cap=15),
               dict(Lq=4, lens=FAKE), dict(ws=None), dict(nws=0), dict(k=FAKE + 4), dict(block=0)):
        assert weight(lib, **kw) == 1, kw
    for kw in (dict(dt=0), dict(d=96), dict(block=48, cap=99), dict(Hq=34)):
        assert weight(lib, **kw) == 2, kw


def test_evict_refusals(lib):
    def select(score=FAKE, B=1, Hkv=2, T=100, n_keep=10, n_sink=4, n_recent=6, keep=FAKE, count=FAKE):
        return lib.spa_evict_select(score, None, B, Hkv, T, n_keep, n_sink, n_recent, keep, count, None)

    for kw in (dict(score=None), dict(keep=None), dict(count=None), dict(B=0), dict(T=0), dict(n_keep=0),
               dict(n_sink=-1), dict(n_recent=-1), dict(n_recent=7)):
        assert select(**kw) == 1, kw

    def gather(kc=FAKE, vc=FAKE, score=FAKE, dt=1, T=100, d=128, n_keep=10, T_out=10, ko=OTHER, vo=OTHER, so=OTHER,
               keep=FAKE):
        return lib.spa_cache_gather(kc, vc, score, dt, 1, 2, T, d, keep, n_keep, None, T_out, ko, vo, so, None)

    for kw in (dict(kc=None), dict(vo=None), dict(score=None), dict(so=None), dict(keep=None), dict(T_out=9),
               dict(dt=3), dict(ko=FAKE), dict(so=FAKE), dict(n_keep=0), dict(kc=FAKE + 8)):
        assert gather(**kw) == 1, kw
    assert gather(d=60) == 2


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    q = torch.zeros((1, 4, 2, 128), dtype=torch.bfloat16)
    f = torch.ones(64, dtype=torch.float64)
    with pytest.raises(ValueError):
        spa.spa_rope(q, None, f)
    with pytest.raises(ValueError):
        spa.spa_sparse_attn_tree(q, q, q, torch.zeros((1, 2), dtype=torch.int32), 16, None, None, 0.1)
    with pytest.raises(ValueError):
        spa.spa_evict_select(torch.zeros((1, 2, 10)), 4)
