"""The selective scan's one wait, run out without a fault: slices whose predecessor has not
run give up after a short limit, report it, and the row stays given up."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
from mamba_ssd_chunked_02_gb300 import layer as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_turns_run_out_report_and_leave_the_context_usable(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    b, T, D, N = 40, 400, 1000, 16
    x, dt = (torch.rand(b, T, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    B, C = (torch.randn(b, T, 1, N, device="cuda", generator=g).to(dtype) for _ in range(2))
    A = -torch.rand(D, N, device="cuda", generator=g)
    need = m2.scan_workspace_size(L.ScanShape(b, T, D, N, 1, m2.BF16 if dtype == torch.bfloat16 else m2.F32, 0))
    space = torch.zeros(need // 4, dtype=torch.int32, device="cuda")
    want, fin = m2.scan_fwd(x, dt, A, B, C)
    assert m2.device_error() == 0
    y = torch.full_like(x, 7.0)
    m2.scan_selftest_turn_timeout(x, dt, A, B, C, y, torch.empty_like(fin), space, limit_us=2000)
    assert m2.device_error() == m2.DEVERR_CHAIN_SCAN
    assert m2.device_error() == 0                          # cleared
    # every row stays given up, although its first slice finished afterwards
    assert (space[:-1] == -1).all()
    # the slices that gave up wrote nothing; the first is right
    kept = (y == 7.0).all(-1).all(0)
    cut = int(kept.int().argmax())
    assert 0 < cut < T and kept[cut:].all() and torch.equal(y[:, :cut], want[:, :cut])
    again, fin2 = m2.scan_fwd(x, dt, A, B, C, workspace=space)
    assert torch.equal(again, want) and torch.equal(fin2, fin) and m2.device_error() == 0
