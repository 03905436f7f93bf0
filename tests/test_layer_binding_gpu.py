"""The Python binding of the layer operators: what it refuses beside test_layer_gpu."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def test_a_width_beyond_32_bits_is_not_cut_down():
    x, w = torch.zeros(1, 2, 0, device="cuda"), torch.zeros(0, (1 << 32) + 4, device="cuda")
    with pytest.raises(m2.Mamba2Error, match="conv_fwd"):
        m2.conv_fwd(x, w)


def test_written_tensors_share_no_memory_with_others():
    b, T, D, N = 2, 12, 16, 8
    x, w = torch.randn(b, T, D, device="cuda"), torch.randn(D, 4, device="cuda")
    window = torch.randn(b, 3, D, device="cuda")
    with pytest.raises(ValueError, match="final_state must not overlap initial_state"):
        m2.conv_fwd(x, w, None, window, final_state=window)     # the window is written before all of it is read
    with pytest.raises(ValueError, match="y must not overlap x"):
        m2.conv_fwd(x, w, y=x)
    with pytest.raises(ValueError, match="y must not overlap x"):
        m2.norm_fwd(x[:, 1:], y=x[:, :-1])
    wide = torch.zeros(b, T, 3 * D, device="cuda")
    with pytest.raises(ValueError, match="y must not overlap x"):
        m2.norm_fwd(wide[:, :, :D], y=wide[:, :, D - 1:2 * D - 1])
    with pytest.raises(ValueError, match="dx must not overlap dy"):
        m2.conv_bwd(x, w, dy=wide[:, :, :D], grads=dict(dx=wide.view(-1)[:x.numel()].view_as(x)))
    one = torch.zeros(D, device="cuda")
    A, B = -torch.ones(D, N, device="cuda"), torch.randn(b, T, 1, N, device="cuda")
    with pytest.raises(ValueError, match="dD must not overlap ddt_bias"):
        m2.scan_bwd(x, x, A, B, B, one, None, one, dy=x, grads=dict.fromkeys(("dD", "ddt_bias"), torch.zeros_like(one)))
    state = torch.zeros(b, D, N, device="cuda")
    with pytest.raises(ValueError, match="state must not overlap x"):
        m2.scan_step(state, state.view(-1)[:b * D].view(b, D), x[:, 0], A, B[:, 0], B[:, 0])
    need = m2.scan_bwd_workspace_size(m2.layer.ScanShape(b, T, D, N, 1, m2.F32, 0))
    space = torch.zeros(need, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace must not overlap dfinal"):
        m2.scan_bwd(x, x, A, B, B, dy=x, dfinal=space.view(torch.float32)[:b * D * N].view(b, D, N), workspace=space)


def test_slices_of_one_buffer_side_by_side_are_fine():
    """x, z and y as columns of one buffer, inputs that are each other, and a tensor of no elements."""
    wide = torch.randn(2, 9, 80, device="cuda")
    x, z, y = wide[:, :, :16], wide[:, :, 16:32], wide[:, :, 32:48]
    want = m2.norm_fwd(x.clone(), None, z.clone())
    assert torch.equal(m2.norm_fwd(x, None, z, y=y), want) and torch.equal(y, want)
    w = torch.randn(16, 4, device="cuda")
    want, fin = m2.conv_fwd(x.clone(), w)
    got, f = m2.conv_fwd(x, w, y=wide[:, :, 64:], final_state=torch.empty_like(fin))
    assert torch.equal(got, want) and torch.equal(f, fin) and torch.equal(wide[:, :, 64:], want)
    half = wide[:, :, :16].contiguous()
    assert torch.equal(m2.norm_fwd(half, None, half), m2.norm_fwd(half, None, half.clone()))
    m2.conv_fwd(x[:, :0], w, y=x[:, :0])


def test_workspaces_of_the_size_asked_for():
    b, T, D, N = 2, 300, 64, 16
    x, w, dy = torch.randn(b, T, D, device="cuda"), torch.randn(D, 4, device="cuda"), torch.randn(b, T, D, device="cuda")
    one, A, B = torch.randn(D, device="cuda"), -torch.ones(D, N, device="cuda"), torch.randn(b, T, 1, N, device="cuda")
    for need, call in (
            (m2.conv_bwd_workspace_size(m2.ConvShape(b, T, D, 4, m2.F32, 1)), lambda s: m2.conv_bwd(x, w, dy=dy, workspace=s)),
            (m2.norm_bwd_workspace_size(m2.NormShape(b, T, D, 1, 1e-5, m2.F32, 0)),
             lambda s: m2.norm_bwd(x, one, dy=dy, workspace=s)),
            (m2.scan_bwd_workspace_size(m2.ScanShape(b, T, D, N, 1, m2.F32, 0)),
             lambda s: m2.scan_bwd(x, x, A, B, B, dy=dy, workspace=s))):
        assert need > 0
        space = torch.empty(need, dtype=torch.uint8, device="cuda")
        got, want = call(space), call(None)
        assert all(torch.equal(got[k], want[k]) for k in want if want[k] is not None)
        with pytest.raises(m2.Mamba2Error, match="workspace"):
            call(space[:-16])
