"""Values at the ends of what e4m3 with a scale can stand for: groups of NaN alone."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
import proj_ref as R
from test_proj_gpu import BF16, F32, INF, NAN, f64, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", ["row", "block"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=("f32", "bf16"))
def test_groups_without_a_finite_value(dt, group):
    """The scale is that of the other values: 2^-127 where there is none, whatever the type."""
    x = torch.full((130, 384), NAN)
    x[:, 256:] = 1.5                  # a group with values beside those without
    x[1, :128:2], x[2, :128:2], x[3, 5] = INF, -INF, -NAN
    x[4, 130:140] = INF
    if group == "row":
        x[5, :128] = 0.25
    v = x.to(dt)
    rows, cols = (1, 128) if group == "row" else (128, 128)
    q, s = m2.quant8(v.cuda(), group=group)
    want = R.quant(f64(v), rows, cols)
    same(s, want[1], "scales")
    same(q, want[0], "q")
