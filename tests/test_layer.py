"""Layer operators on the host (no GPU): the fp64 gradients the GPU tests compare with,
against central differences of the fp64 forward; and the C ABI's refusals."""
import ctypes

import pytest
import torch

import layer_ref as R
import mamba_ssd_chunked_02_gb300 as m2
from mamba_ssd_chunked_02_gb300 import build as m2build
from mamba_ssd_chunked_02_gb300 import layer as L


def _differences(loss, inputs, grads, h=1e-5):
    """Every element of every gradient against (f(v + h) - f(v - h)) / 2h.  The third
    derivatives here are below 1e2 of the loss's scale, so h = 1e-5 leaves 1e-8 of
    truncation and 1e-10 of rounding."""
    for name, v in inputs.items():
        flat, want = v.view(-1), grads["d" + name].reshape(-1)
        for k in range(flat.numel()):
            keep = flat[k].item()
            flat[k] = keep + h
            up = loss()
            flat[k] = keep - h
            down = loss()
            flat[k] = keep
            got = (up - down) / (2 * h)
            assert abs(got - want[k]) <= 1e-6 * (1 + abs(got)), (name, k, got.item(), want[k].item())


def _rand(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, dtype=torch.float64) * scale


@pytest.mark.parametrize("W,act,lengths", [(2, True, None), (4, False, [5, 1]), (3, True, [0, 4])])
def test_conv_gradient_against_differences(W, act, lengths):
    g = torch.Generator().manual_seed(1)
    b, T, D = 2, 5, 3
    v = dict(x=_rand(g, b, T, D), w=_rand(g, D, W), bias=_rand(g, D), init=_rand(g, b, W - 1, D))
    dy, df = _rand(g, b, T, D), _rand(g, b, W - 1, D)

    def loss():
        y, f = R.conv(v["x"], v["w"], v["bias"], v["init"], lengths, act)
        return (y * dy).sum() + (f * df).sum()

    _differences(loss, v, R.conv(v["x"], v["w"], v["bias"], v["init"], lengths, act, dy, df))


@pytest.mark.parametrize("G,gate,softplus,lengths", [(1, True, True, None), (2, False, True, [4, 0]),
                                                     (2, True, False, [2, 4])])
def test_scan_gradient_against_differences(G, gate, softplus, lengths):
    g = torch.Generator().manual_seed(2)
    b, T, D, N = 2, 4, 4, 3
    v = dict(x=_rand(g, b, T, D), dt=_rand(g, b, T, D, scale=0.5) + (0 if softplus else 1), A=-_rand(g, D, N).abs(),
             B=_rand(g, b, T, G, N), C=_rand(g, b, T, G, N), D=_rand(g, D), dt_bias=_rand(g, D, scale=0.1),
             init=_rand(g, b, D, N))
    if gate:
        v["z"] = _rand(g, b, T, D)
    dy, df = _rand(g, b, T, D), _rand(g, b, D, N)

    def args():
        return (v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v.get("z"), v["dt_bias"], v["init"], lengths, softplus)

    def loss():
        y, f = R.scan(*args())
        return (y * dy).sum() + (f * df).sum()

    _differences(loss, v, R.scan(*args(), dy, df))


@pytest.mark.parametrize("G,gate", [(1, "first"), (2, "after"), (3, None)])
def test_norm_gradient_against_differences(G, gate):
    g = torch.Generator().manual_seed(3)
    v = dict(x=_rand(g, 2, 2, 6), w=_rand(g, 6))
    if gate:
        v["z"] = _rand(g, 2, 2, 6)
    dy = _rand(g, 2, 2, 6)
    first = gate != "after"
    _differences(lambda: (R.norm(v["x"], v["w"], v.get("z"), G, 1e-3, first) * dy).sum(), v,
                 R.norm(v["x"], v["w"], v.get("z"), G, 1e-3, first, dy))


# ---- refusals of the C ABI: everything is checked before the first CUDA call --------------------

@pytest.fixture(scope="module")
def lib():
    m2build.build()
    return m2.load()


P = 1 << 20       # an aligned address that is never read


def _conv(**kw):
    s = dict(batch=2, seqlen=4, channels=8, width=4, dtype=m2.BF16, flags=L.CONV_SILU)
    s.update(kw)
    return L.ConvShape(**s)


def _scan(**kw):
    s = dict(batch=2, seqlen=4, channels=8, states=16, groups=1, dtype=m2.BF16, flags=L.SCAN_SOFTPLUS)
    s.update(kw)
    return L.ScanShape(**s)


def _norm(**kw):
    s = dict(batch=2, seqlen=4, channels=8, groups=1, eps=1e-5, dtype=m2.BF16, flags=0)
    s.update(kw)
    return L.NormShape(**s)


def _status(name, shape, ptrs, strides=None, space=None):
    tail = [None, 0, None] if space == "none" else [P, 1 << 40, None] if space else [None]
    at = ctypes.addressof(strides) if strides is not None else None
    return L._fn(name)(ctypes.addressof(shape) if shape is not None else None, at, *ptrs, *tail)


def test_conv_refusals(lib):
    ok = [P] * 7
    assert _status("conv_fwd", None, ok) == m2.ERR_INVALID_ARG
    for bad in (dict(batch=-1), dict(seqlen=-1), dict(channels=-1), dict(dtype=5), dict(flags=2), dict(width=0)):
        assert _status("conv_fwd", _conv(**bad), ok) == m2.ERR_INVALID_ARG
    for bad in (dict(width=1), dict(width=5), dict(seqlen=1 << 31), dict(channels=1 << 25)):
        assert _status("conv_fwd", _conv(**bad), ok) == m2.ERR_UNSUPPORTED
    for k in (0, 1, 5):      # x, w, y are required
        assert _status("conv_fwd", _conv(), ok[:k] + [None] + ok[k + 1:]) == m2.ERR_INVALID_ARG
    assert _status("conv_fwd", _conv(), [P + 1] + ok[1:]) == m2.ERR_INVALID_ARG
    st = L._strides2(32, 8, 32, 4)      # y's tokens would overlap
    assert _status("conv_fwd", _conv(), ok, st) == m2.ERR_INVALID_ARG
    st = L._strides2(-32, 8, 32, 8)
    assert _status("conv_fwd", _conv(), ok, st) == m2.ERR_INVALID_ARG
    assert _status("conv_step", _conv(), [P] * 5) == m2.ERR_INVALID_ARG       # seqlen is not 1
    assert _status("conv_step", _conv(seqlen=1), [None] + [P] * 4) == m2.ERR_INVALID_ARG
    assert L._fn("conv_bwd_ws")(ctypes.addressof(_conv(width=9))) == 0
    assert _status("conv_bwd", _conv(), [P] * 11, space="none") == m2.ERR_WORKSPACE
    assert _status("conv_bwd", _conv(), [P] * 8 + [None] + [P] * 2, space=True) == m2.ERR_INVALID_ARG   # dw


def test_scan_refusals(lib):
    ok = [P] * 12
    for bad in (dict(batch=-1), dict(groups=0), dict(groups=3), dict(states=0), dict(flags=4), dict(dtype=-1)):
        assert _status("scan_fwd", _scan(**bad), ok, space=True) == m2.ERR_INVALID_ARG
    for bad in (dict(states=12), dict(states=256), dict(seqlen=1 << 31),
                dict(channels=1 << 24, groups=1 << 21, states=16)):
        assert _status("scan_fwd", _scan(**bad), ok, space=True) == m2.ERR_UNSUPPORTED
    for k in (0, 1, 2, 3, 4, 10, 11):
        assert _status("scan_fwd", _scan(), ok[:k] + [None] + ok[k + 1:], space=True) == m2.ERR_INVALID_ARG
    long = _scan(batch=1, seqlen=65536)
    assert L.scan_workspace_size(long) > 0
    assert _status("scan_fwd", long, ok, space="none") == m2.ERR_WORKSPACE
    assert L.scan_workspace_size(_scan(states=5)) == 0 and L.scan_bwd_workspace_size(_scan(groups=0)) == 0
    assert _status("scan_step", _scan(), [P] * 10) == m2.ERR_INVALID_ARG
    assert _status("scan_step", _scan(seqlen=1), [P + 2] + [P] * 9) == m2.ERR_INVALID_ARG
    assert _status("scan_bwd", _scan(), [P] * 21, space="none") == m2.ERR_WORKSPACE
    for k in (12, 13, 14, 15, 16, 17, 18, 19):      # dx .. ddt_bias (D, z and dt_bias are given)
        p = [P] * 21
        p[k] = None
        assert _status("scan_bwd", _scan(), p, space=True) == m2.ERR_INVALID_ARG


def test_norm_refusals(lib):
    ok = [P] * 4
    for bad in (dict(groups=0), dict(groups=3), dict(eps=-1.0), dict(eps=float("nan")), dict(flags=2), dict(dtype=9)):
        assert _status("norm_fwd", _norm(**bad), ok) == m2.ERR_INVALID_ARG
    assert _status("norm_fwd", _norm(), [None] + ok[1:]) == m2.ERR_INVALID_ARG
    assert _status("norm_bwd", _norm(), [P] * 7, space="none") == m2.ERR_WORKSPACE
    assert _status("norm_bwd", _norm(), [P] * 5 + [None, P], space=True) == m2.ERR_INVALID_ARG    # dz


def test_exports_and_python_refusals(lib):
    for n in L.SYMBOLS:
        assert hasattr(lib, n)
    x = torch.zeros(1, 2, 8)
    with pytest.raises(ValueError, match="no CPU path"):
        m2.conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        m2.norm_fwd(x.half())
    with pytest.raises(TypeError, match="torch.Tensor"):
        m2.scan_fwd(None, None, None, None, None)
