"""Projection operators on the host (no GPU): refusals beside test_proj.py's."""
import pytest

import mamba_ssd_chunked_02_gb300 as m2
from mamba_ssd_chunked_02_gb300 import build as m2build
from test_proj import P, SIZE, _call, _longs, _proj


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
