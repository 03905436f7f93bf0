"""Layer operators past 2^31 elements: strides that lead there, and outputs that are that long.

A strided call takes the kernels of the same call on contiguous tensors (all strides are
multiples of 16 bytes), so its results are equal bit for bit.  The end of a long bf16 call is compared
with a short fp32 call on its last tokens, which starts from the state the long one had there; bounds
as in test_layer_gpu."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
from test_layer_gpu import BF16, close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    yield
    torch.cuda.empty_cache()


def rand(*shape, scale=1.0):
    return (torch.randn(*shape, device="cuda") * scale).to(BF16)


@pytest.mark.parametrize("b,T,sb,st", [(3, 20, (1 << 31) + 16, 64), (2, 70, 64, (1 << 26) + 128)], ids=["far rows", "far tokens"])
def test_strides_beyond_32_bits(b, T, sb, st):
    torch.manual_seed(1)
    D, N = 64, 16
    flat = torch.empty((b - 1) * sb + (T - 1) * st + D, dtype=BF16, device="cuda")
    flat2 = torch.empty_like(flat)

    def far(v, buf=flat):
        out = buf.as_strided(v.shape, (sb, st, 1) if v.dim() == 3 else (sb, st, N, 1))
        return out.copy_(v)

    x, z, dy, dt = (rand(b, T, D) for _ in range(4))
    w, scale, A = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda"), -torch.rand(D, N, device="cuda")
    B, C = rand(b, T, 1, N), rand(b, T, 1, N)
    out = flat2.as_strided((b, T, D), (sb, st, 1))
    want, fin = m2.conv_fwd(x, w)
    got, f = m2.conv_fwd(far(x), w, y=out)
    assert torch.equal(got, want) and torch.equal(f, fin)
    assert torch.equal(m2.norm_fwd(far(x), scale, z, y=out), m2.norm_fwd(x, scale, z))
    want, fin = m2.scan_fwd(x, dt, A, B, C, dt_softplus=True)
    for name in ("x", "dt", "B", "C"):
        t = dict(x=x, dt=dt, B=B, C=C)
        t[name] = far(t[name])
        got, f = m2.scan_fwd(t["x"], t["dt"], A, t["B"], t["C"], dt_softplus=True, y=out)
        assert torch.equal(got, want) and torch.equal(f, fin), name
    for op, args in ((m2.conv_bwd, dict(x=x, w=w, dy=dy)), (m2.norm_bwd, dict(x=x, w=scale, z=z, dy=dy)),
                     (m2.scan_bwd, dict(x=x, dt=dt, A=A, B=B, C=C, z=z, dy=dy))):
        want = op(**args)
        for name in args:
            if args[name].dtype == BF16:
                got = op(**{**args, name: far(args[name])})
                assert all(torch.equal(got[k], want[k]) for k in want if want[k] is not None), (op.__name__, name)


T, D, TAIL = 560_000, 4096, 96       # 2.3e9 elements


def test_long_norm_and_conv():
    torch.manual_seed(2)
    x, dy = torch.empty(1, T, D, dtype=BF16, device="cuda").normal_(), torch.empty(1, T, D, dtype=BF16, device="cuda").normal_()
    w, scale = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    end = [v[:, -TAIL:].contiguous() for v in (x, dy)]
    wide = [v.float() for v in end]
    y = m2.norm_fwd(x, scale, dy)
    assert torch.equal(y[:, -TAIL:], m2.norm_fwd(end[0], scale, end[1]))
    g = m2.norm_bwd(x, scale, dy, dy)
    want = m2.norm_bwd(wide[0], scale, wide[1], wide[1])
    for k in ("dx", "dz"):
        close(g[k][:, -TAIL:], want[k].cpu(), k)
    del y, g
    window = x[:, -TAIL - 3:-TAIL].contiguous()
    y, fin = m2.conv_fwd(x, w)
    want, f = m2.conv_fwd(end[0], w, None, window)
    assert torch.equal(y[:, -TAIL:], want) and torch.equal(fin, f)
    del y
    g = m2.conv_bwd(x, w, dy=dy)
    close(g["dx"][:, -TAIL:], m2.conv_bwd(wide[0], w, None, window.float(), dy=wide[1])["dx"].cpu(), "dx")


def test_long_scan():
    torch.manual_seed(3)
    N = 8
    x, dy = torch.empty(1, T, D, dtype=BF16, device="cuda").normal_(), torch.empty(1, T, D, dtype=BF16, device="cuda").normal_()
    dt = torch.empty(1, T, D, dtype=BF16, device="cuda").normal_()
    A, B, C = -torch.rand(D, N, device="cuda") - 0.1, rand(1, T, 1, N), rand(1, T, 1, N)
    at = T - TAIL
    _, state = m2.scan_fwd(x[:, :at], dt[:, :at], A, B[:, :at], C[:, :at], dt_softplus=True)
    end = [v[:, at:].float().contiguous() for v in (x, dt, B, C, dy)]
    y, fin = m2.scan_fwd(x, dt, A, B, C, dt_softplus=True)
    want, f = m2.scan_fwd(end[0], end[1], A, end[2], end[3], None, None, None, state, dt_softplus=True)
    close(y[:, at:], want.cpu(), "y")
    close(fin, f.cpu(), "final_state")
    del y
    g = m2.scan_bwd(x, dt, A, B, C, dy=dy, dt_softplus=True)
    want = m2.scan_bwd(end[0], end[1], A, end[2], end[3], None, None, None, state, end[4], dt_softplus=True)
    for k in ("dx", "ddt", "dB", "dC"):
        close(g[k][:, at:], want[k].cpu(), k)
