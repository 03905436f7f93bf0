"""Values at the ends of what e4m3 with a scale can stand for: groups of NaN alone, and operands whose
values are beyond fp32."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
import proj_ref as R
from test_proj_gpu import BF16, E4M3, F32, INF, NAN, f64, same

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


@pytest.mark.parametrize("K", [64, 131])
@pytest.mark.parametrize("low,high", [(90, 121), (100, 128), (-127, 128)])
def test_scales_beyond_fp32_turned(low, high, K):
    """x along its columns for dw where values pass fp32's largest (an fp32 maximum rounds up to 2^128;
    scales go to 2^127): every e4m3 number, read off with one row of dy a tile, small enough for the
    product to be one that fp32 holds."""
    r = torch.Generator().manual_seed(41)
    M = 300
    bits = torch.randint(0, 256, (M, K), generator=r).to(torch.uint8)
    bits[(bits & 127) == 127] = 5
    bits[:, 3] = 0x7e                                  # 448 throughout
    bits[::17] = 128
    e = torch.randint(low, high, (M, 1), generator=r)
    e[::17] = -127
    e[5] = high - 1
    room = torch.zeros(M, -(-K // 16) * 16, dtype=torch.uint8, device="cuda")
    room[:, :K] = bits.cuda()
    q = room.view(E4M3)[:, :K]
    s = (e.expand(M, -(-K // 128)) + 127).to(torch.uint8).cuda().view(torch.float8_e8m0fnu)
    want = R.dequant(*R.quant(bits.view(E4M3).double() * 2.0 ** e.double(), 128, 1), 128, 1)
    wq, ws = m2.quant8(torch.ones(3, K, device="cuda"), group="block")
    for row in (1, 5, 130, 299):
        dy = torch.zeros(M, 3)
        dy[row, 1] = 2.0 ** -60
        dw = m2.proj8_bwd(dy.cuda(), q, s, wq, ws, need_dx=False)["dw"]
        assert (dw[0] == 0).all() and (dw[2] == 0).all()
        exact = want[row].abs() >= 2.0 ** -66          # the product is a normal fp32 number
        assert torch.equal(f64(dw[1])[exact], want[row][exact] * 2.0 ** -60), row


def test_largest_fp32_values_through_quant8_and_the_gradient():
    """fp32's largest number rounds to 256 * 2^120 = 2^128."""
    x = torch.full((130, 128), torch.finfo(F32).max)
    x[1:] *= 0.25
    (q, s), (wq, ws) = m2.quant8(x.cuda()), m2.quant8(torch.ones(2, 128, device="cuda"), group="block")
    assert f64(q[0, 0]).item() * f64(s[0, 0]).item() == 2.0 ** 128
    dy = torch.zeros(130, 2)
    dy[0, 0], dy[1, 1] = 2.0 ** -10, 2.0 ** -10
    dw = m2.proj8_bwd(dy.cuda(), q, s, wq, ws, need_dx=False)["dw"]
    assert (dw[0] == 2.0 ** 118).all() and (dw[1] == 2.0 ** 116).all()


def test_a_scale_that_is_not_a_number_turned():
    """The byte 255 is e8m0's NaN: every value of the group is NaN, for dw as for the product; the
    other rows' scale is theirs."""
    x = torch.ones(256, 256)
    q, s = m2.quant8(x.cuda())
    s.view(torch.uint8)[7, 1] = 255
    wq, ws = m2.quant8(torch.ones(2, 256, device="cuda"), group="block")
    y = m2.proj8_fwd(q, s, wq, ws)
    assert y[7].isnan().all() and (y[:7] == 256).all() and (y[8:] == 256).all()
    dy = torch.ones(256, 2)
    dw = m2.proj8_bwd(dy.cuda(), q, s, wq, ws, need_dx=False)["dw"]
    assert (dw[:, :128] == 256).all() and dw[:, 128:].isnan().all()
