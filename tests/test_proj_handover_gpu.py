"""The accumulators' way between the two blocks of a pair: products of one or two contracted blocks,
where a tile's sums are handed back to the issuing block, and the next one's begin, every few
microseconds.  Whole numbers, so that every sum is exact and every bit of both blocks' rows is known;
each form of the product many times over."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
from test_proj_gpu import BF16, F32

pytestmark = pytest.mark.gpu


def whole(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-4, 5, shape, device="cuda", generator=g).float()
    v[::50, 0] = 7.0                      # the same scale for all groups that have it; others are exact too
    return v


@pytest.mark.parametrize("M,K,N", [(9000, 128, 2500), (9000, 100, 2504), (30000, 256, 333), (4000, 129, 8000)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=("f32", "bf16"))
def test_short_sums_forward(M, K, N, dt):
    x, w = whole(M, K, seed=1), whole(N, K, seed=2)
    ops = (*m2.quant8(x), *m2.quant8(w, group="block"))
    want = (x.double() @ w.double().t()).to(dt)
    y = torch.empty(M, N, device="cuda", dtype=dt)
    for _ in range(60):
        y.fill_(float("nan"))
        m2.proj8_fwd(*ops, y=y)
        assert torch.equal(y, want)
    assert m2.device_error() == 0


@pytest.mark.parametrize("M,K,N", [(9000, 2560, 128), (9000, 2500, 200), (130, 5000, 3000), (256, 2504, 7000)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=("f32", "bf16"))
def test_short_sums_of_gradients(M, K, N, dt):
    """dx with one or two blocks of outputs, dw with one or two of tokens (and the other with many)."""
    x, w, dy = whole(M, K, seed=3), whole(N, K, seed=4), whole(M, N, seed=5)
    ops = (*m2.quant8(x), *m2.quant8(w, group="block"))
    dx, dw = (dy.double() @ w.double()).to(dt), (dy.double().t() @ x.double()).float()
    g = m2.proj8_bwd(dy.to(dt), *ops)
    for _ in range(30):
        for t in (g["dx"], g["dw"]):
            t.fill_(float("nan"))
        m2.proj8_bwd(dy.to(dt), *ops, grads=g)
        assert torch.equal(g["dx"], dx) and torch.equal(g["dw"], dw)
    assert m2.device_error() == 0
