"""Layer operators on the host (no GPU): refusals and host-side paths beside test_layer."""
import ctypes

import pytest

import mamba_ssd_chunked_02_gb300 as m2
from mamba_ssd_chunked_02_gb300 import build as m2build
from mamba_ssd_chunked_02_gb300 import layer as L

P = 1 << 20       # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    m2build.build()
    return m2.load()


def test_turn_selftest_refusals(lib):
    f = L._fn("scan_selftest")

    def status(shape, ptrs=(P,) * 8, space=1 << 40, limit=1000):
        return f(ctypes.addressof(shape), *ptrs, space, limit, None)

    turns = L.ScanShape(40, 400, 1000, 16, 1, m2.BF16, 0)     # 1280 rows of blocks
    assert status(turns, limit=0) == m2.ERR_INVALID_ARG and status(turns, limit=100001) == m2.ERR_INVALID_ARG
    assert status(L.ScanShape(2, 400, 1000, 16, 1, m2.BF16, 0)) == m2.ERR_UNSUPPORTED
    assert status(L.ScanShape(40, 400, 1000, 12, 1, m2.BF16, 0)) == m2.ERR_UNSUPPORTED
    for k in range(7):
        assert status(turns, [None if i == k else P for i in range(8)]) == m2.ERR_INVALID_ARG
    assert status(turns, space=4) == m2.ERR_WORKSPACE
