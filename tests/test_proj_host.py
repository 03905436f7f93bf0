"""Projection operators on the host (no GPU): refusals beside test_proj.py's."""
import ctypes

import pytest

import mamba_ssd_chunked_02_gb300 as m2
from mamba_ssd_chunked_02_gb300 import build as m2build
from test_proj import P, SIZE, _call, _longs, _norm, _proj


@pytest.fixture(scope="module")
def lib():
    m2build.build()
    return m2.load()


def test_gradient_pitches(lib):
    """dy's rows may overlap, but step forward; those of x and w may not."""
    back = [P] * 7                        # dy, x, scales, w, scales, dx, dw
    for p in (_longs(16, 32, 8), _longs(32, 16, 8), _longs(0, 32, 8), _longs(32, 32, -1), _longs(32, 32, 1 << 40)):
        assert _call(lib, "proj8_bwd", _proj(), p, *back, *SIZE) == m2.ERR_INVALID_ARG
    # a pitch of dy of 0 is taken: the workspace is what is missing here
    assert _call(lib, "proj8_bwd", _proj(), _longs(32, 32, 0), *back, None, 0, None) == m2.ERR_WORKSPACE


def test_timeout_selftest_refusals(lib):
    ok = [P] * 5                          # x, scales, w, scales, y

    f = lib.mamba2_proj8_selftest_timeout
    f.restype = ctypes.c_int

    def status(shape=None, ptrs=ok, limit=1000):
        return f(ctypes.byref(shape or _proj()), *(ctypes.c_void_p(p) for p in ptrs), ctypes.c_uint32(limit), None)

    assert status(limit=0) == m2.ERR_INVALID_ARG and status(limit=100001) == m2.ERR_INVALID_ARG
    for bad in (dict(tokens=0), dict(outputs=0), dict(tokens=-1), dict(dtype=5), dict(flags=1)):
        assert status(_proj(**bad)) == m2.ERR_INVALID_ARG
    assert status(_proj(inputs=0)) == m2.ERR_UNSUPPORTED
    for k in range(5):
        assert status(ptrs=[None if i == k else P for i in range(5)]) == m2.ERR_INVALID_ARG
    for k in (0, 2):
        assert status(ptrs=[P + 8 if i == k else P for i in range(5)]) == m2.ERR_INVALID_ARG


def test_strides_of_x_are_not_looked_at_in_add_norm_s_gradient(lib):
    """It has no x: what the strides say of one is not checked (the workspace is what is missing here)."""
    back = [P] * 7                        # total, w, dy, dtotal, dx, dresidual, dw
    for x in ((-1, 5), (1 << 50, -7)):
        st = _longs(*x, 128, 32, 128, 32, 128, 32)
        assert _call(lib, "add_norm_bwd", _norm(), st, *back, None, 0, None) == m2.ERR_WORKSPACE
    for k in (2, 4, 6):
        bad = [128, 32] * 4
        bad[k] = -1
        assert _call(lib, "add_norm_bwd", _norm(), _longs(*bad), *back, *SIZE) == m2.ERR_INVALID_ARG
