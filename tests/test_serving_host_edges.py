"""More refusals of the serving operators. CPU only: every refused call fails a host
check before any launch."""
from tests.test_serving_host import FAKE, lib, weight  # noqa: F401  (lib: the fixture)


def test_weight_refuses_fp32_tensors_off_their_elements(lib):  # noqa: F811
    for kw in (dict(lse=FAKE + 2), dict(out=FAKE + 2), dict(lse=FAKE + 1)):
        assert weight(lib, **kw) == 1, kw
