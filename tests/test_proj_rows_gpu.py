"""Distances between the rows of the 8-bit product's tensors: gradients that are one row for many
tokens, and rows that lie in one another."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
from test_proj_gpu import BF16, F32, Gen, _operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16], ids=("f32", "bf16"))
@pytest.mark.parametrize("M,N", [(300, 200), (300, 90), (5, 130), (4000, 1000)])
def test_gradient_of_a_broadcast_row(M, N, dt):
    """dy expanded over the tokens (stride 0) is read in place, as add_norm and quant8 read such."""
    ops, _, _ = _operands(M, 260, N)
    row = Gen(1).randn(1, N, dtype=dt).cuda()
    want = m2.proj8_bwd(row.expand(M, N).contiguous(), *ops)
    got = m2.proj8_bwd(row.expand(M, N), *ops)
    assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dw"], want["dw"])
    deep = [ops[0].unflatten(0, (M // 5, 5)), ops[1].unflatten(0, (M // 5, 5)), *ops[2:]]
    got = m2.proj8_bwd(row[None].expand(M // 5, 5, N), *deep)
    assert torch.equal(got["dx"].flatten(0, 1), want["dx"]) and torch.equal(got["dw"], want["dw"])


def test_rows_that_overlap_each_other():
    """Distances between rows that lie within one another: read where the operands need no copy's map
    (dy), refused by name elsewhere."""
    (q, s, wq, ws), _, _ = _operands(6, 200, 40)
    buf = Gen(2).randn(600).cuda()
    dy = buf.as_strided((6, 40), (8, 1))
    got, want = m2.proj8_bwd(dy, q, s, wq, ws), m2.proj8_bwd(dy.contiguous(), q, s, wq, ws)
    assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dw"], want["dw"])
    with pytest.raises(ValueError, match="x: rows must not overlap"):
        m2.proj8_fwd(q[:1].expand(6, 200), s, wq, ws)
    with pytest.raises(ValueError, match="w: rows must not overlap"):
        m2.proj8_fwd(q, s, wq[:1].expand(40, 200), ws)
    with pytest.raises(ValueError, match="y: rows must not overlap"):
        m2.proj8_fwd(q, s, wq, ws, y=torch.empty(1, 40, device="cuda").expand(6, 40))
    with pytest.raises(ValueError, match="dy: tokens must lie at even distances"):
        m2.proj8_bwd(torch.zeros(2, 4, 40, device="cuda")[:, :3], q.view(2, 3, 200), s.view(2, 3, 2), wq, ws)
