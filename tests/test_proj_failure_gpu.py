"""The 8-bit product's waits, run out without a fault: one block of each cluster keeps its scales
back, for which the tensor cores' warp of its pair then waits in vain; the other blocks find out, what
is in flight lands, and every block ends."""
import time

import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2

pytestmark = pytest.mark.gpu


# few rows: a lone block, clusters, more operands than stages; pairs with one tile each and with several, of
# 224 and 128 columns; several pairs a tile
@pytest.mark.parametrize("M,K,N", [(1, 128, 128), (1, 1024, 128), (20, 2560, 2560), (100, 5120, 2560), (3, 32768, 64),
                                   (300, 256, 512), (9000, 512, 4000), (20000, 2048, 96), (256, 8192, 256),
                                   (500, 4096, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=("bf16", "f32"))
def test_a_wait_that_runs_out_is_reported_and_the_context_stays_usable(M, K, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(n, K, device="cuda", generator=g) for n in (M, N))
    ops = (*m2.quant8(x), *m2.quant8(w, group="block"))
    want = m2.proj8_fwd(*ops, dtype=dtype)
    assert m2.device_error() == 0
    y = torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    t = time.time()
    m2.proj8_selftest_timeout(*ops, y, limit_us=2000)
    torch.cuda.synchronize()
    assert time.time() - t < 1.0           # six limits, and what a launch takes
    assert m2.device_error() == m2.DEVERR_TIMEOUT_PROJ8
    assert m2.device_error() == 0          # cleared
    assert (y == 7.0).all()
    # the next calls find all as it should be: tensor memory is free, no barrier or copy is left over
    for _ in range(3):
        assert torch.equal(m2.proj8_fwd(*ops, dtype=dtype), want)
    dy = want.to(torch.bfloat16)
    a, b = m2.proj8_bwd(dy, *ops), m2.proj8_bwd(dy, *ops)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"]) and a["dw"].isfinite().all()
    assert m2.device_error() == 0


def test_a_captured_call_and_a_short_limit():
    """Behind one another in a graph, and each replay reports anew."""
    ops = (*m2.quant8(torch.ones(300, 256, device="cuda")), *m2.quant8(torch.ones(512, 256, device="cuda"), group="block"))
    y, z = torch.full((300, 512), 7.0, device="cuda"), torch.zeros(300, 512, device="cuda")
    m2.proj8_fwd(*ops, y=z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m2.proj8_selftest_timeout(*ops, y, limit_us=1)
        m2.proj8_fwd(*ops, y=z)
    for _ in range(2):
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert m2.device_error() == m2.DEVERR_TIMEOUT_PROJ8
        assert (y == 7.0).all() and (z == 256.0).all()
