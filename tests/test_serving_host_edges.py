"""More refusals of the serving operators. CPU only: every refused call fails a host
check before any launch."""
import ctypes

from tests.test_serving_host import FAKE, OTHER, append, freqs, lib, rope, weight  # noqa: F401  (lib: the fixture)


def test_weight_refuses_fp32_tensors_off_their_elements(lib):  # noqa: F811
    for kw in (dict(lse=FAKE + 2), dict(out=FAKE + 2), dict(lse=FAKE + 1)):
        assert weight(lib, **kw) == 1, kw


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("l", ctypes.c_int64)]


def test_outputs_that_overlap_are_refused(lib):  # noqa: F811
    # the rotated queries and keys, the two caches
    assert rope(lib, ko=OTHER, qo=OTHER) == 1
    assert append(lib, kc=OTHER, vc=OTHER) == 1
    assert append(lib, kc=OTHER, vc=OTHER + 100 * 2 * 128 * 2 - 16) == 1
    # the smaller cache: with the cache, its parts with one another, by one row
    size = 2 * 100 * 128 * 2                                       # bytes of kc: [1, 2, 100, 128] bf16
    far = 0x1000000

    def gather(kc=FAKE, vc=FAKE + far, ko=FAKE + 2 * far, vo=FAKE + 3 * far, score=FAKE + 4 * far, so=FAKE + 5 * far):
        return lib.spa_cache_gather(kc, vc, score, 1, 1, 2, 100, 128, FAKE, 10, None, 10, ko, vo, so, None)

    out = 2 * 10 * 128 * 2
    for kw in (dict(ko=FAKE + size - 256), dict(vo=FAKE + size - 256), dict(ko=FAKE + far - out + 256),
               dict(vo=FAKE + far + 256), dict(vo=FAKE + 2 * far), dict(vo=FAKE + 2 * far + out - 256),
               dict(so=FAKE + 4 * far + 796), dict(so=FAKE + 4 * far)):
        assert gather(**kw) == 1, kw


def test_weight_refuses_an_output_that_overlaps_prev_in_part(lib):  # noqa: F811
    need = lib.spa_attn_weight_workspace_bytes(1, 2, 1, 256, 0)
    far = 0x1000000
    for out in (far + 4, far - 4, far + 2 * 256 * 4 - 4):
        assert lib.spa_attn_weight(FAKE, FAKE, 1, 1, 8, 2, 1, 256, 128, FAKE, None, 128, None, 0, None, 0.1,
                                   FAKE + far, 1.0, FAKE, need, FAKE + out, None) == 1


def test_broadcast_outputs_are_refused(lib):  # noqa: F811
    def call(qo, ko):
        strides = [s and ctypes.byref(Strides(*s)) for s in (qo, ko)]
        return lib.spa_rope(FAKE, None, OTHER, strides[0], FAKE, None, OTHER + 0x100000, strides[1], 1, 2, 4, 2, 8, 128,
                            128, 0, freqs(64), 1.0, None, 0, 0, None)

    for bad in ((0, 1024, 128), (4096, 0, 128), (4096, 1024, 0)):
        assert call(bad, None) == 1 and call(None, bad) == 1
    assert lib.spa_rope_append(FAKE, None, OTHER, ctypes.byref(Strides(512, 0, 128)), FAKE, None, FAKE, None,
                               0x100000, 0x200000, 1, 1, 4, 2, 1, 100, 128, 64, 0, freqs(64), 1.0, None, None, 0,
                               None) == 1


def test_sizes_beyond_the_launch_and_the_index_arithmetic_are_refused(lib):  # noqa: F811
    # 37.5 million blocks: more rows than a grid has; a T that is rounded up past 32 bits
    T = 600_000_000
    assert weight(lib, Hkv=1, T=T, d=64, cap=T // 16) == 2
    assert lib.spa_evict_select(FAKE, None, 1, 1, 2 ** 31 - 1, 10, 4, 6, OTHER, OTHER + 4096, None) == 2
