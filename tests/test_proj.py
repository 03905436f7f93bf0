"""Projection operators on the host (no GPU): the fp64 references, and the C ABI's and the
binding's refusals."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
import proj_ref as R
from mamba_ssd_chunked_02_gb300 import build as m2build
from mamba_ssd_chunked_02_gb300 import proj as L


def test_e4m3_reference_against_all_numbers():
    """Every e4m3 number is itself; midpoints of neighbours go to the even one; a little beside
    them to the nearer one."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(R.e4m3(v), v) and torch.equal(R.e4m3(-v), -v)
    mid = (v[1:] + v[:-1]) / 2
    even = torch.where(torch.arange(126) % 2 == 0, v[:-1], v[1:])
    assert torch.equal(R.e4m3(mid), even)
    assert torch.equal(R.e4m3(mid * (1 + 1e-9)), v[1:]) and torch.equal(R.e4m3(mid * (1 - 1e-9)), v[:-1])


@pytest.mark.parametrize("top,e", [(0.0, -127), (448.0, 0), (448.1, 1), (449.0, 1), (224.0, -1), (1.75, -8), (1.7500001, -7),
                                   (2.0 ** -130, -127), (3e38, 119 + 1)])
def test_scale_exponent(top, e):
    assert R.scale_exponent(top) == e


def test_add_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    t, w, dy, dt = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((2, 3, 5), (5,), (2, 3, 5), (2, 3, 5)))
    dx, dw = R.add_norm_bwd(t, w, 1e-3, dy, dt)

    def loss():
        return (R.add_norm(t, w, 1e-3) * dy).sum() + (t * dt).sum()

    for v, want in ((t, dx), (w, dw)):
        flat, want = v.view(-1), want.reshape(-1)
        for k in range(flat.numel()):
            keep, h = flat[k].item(), 1e-5
            flat[k] = keep + h
            up = loss()
            flat[k] = keep - h
            down = loss()
            flat[k] = keep
            got = (up - down) / (2 * h)
            assert abs(got - want[k]) <= 1e-6 * (1 + abs(got))


def test_proj_gradient_is_that_of_the_rounded_values():
    """Where every value is its own e4m3 number the 8-bit gradients are autograd's."""
    g = torch.Generator().manual_seed(2)
    x, w, dy = (torch.randint(-4, 5, s, generator=g).double() for s in ((5, 7), (3, 7), (5, 3)))
    xx, ww = x.clone().requires_grad_(), w.clone().requires_grad_()
    want = torch.autograd.grad(xx @ ww.t(), [xx, ww], dy)
    for got, ref in zip(R.proj_bwd(dy, x, w), want):
        assert torch.equal(got, ref)


# ---- refusals of the C ABI: everything is checked before the first CUDA call --------------------

@pytest.fixture(scope="module")
def lib():
    m2build.build()
    return m2.load()


P = 1 << 20       # an aligned address that is never read
SIZE = (P, 1 << 40, None)
NO_SPACE = (None, 0, None)


class _Quant8Shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


def _call(lib, name, shape, extra, *args):
    f = getattr(lib, "mamba2_" + name)
    f.restype = ctypes.c_int
    at = [ctypes.byref(s) if s is not None else None for s in (shape, extra)]
    return f(*at, *(ctypes.c_size_t(a) if isinstance(a, int) else a for a in args))


def _norm(**kw):
    s = dict(batch=2, seqlen=4, channels=32, eps=1e-5, dtype=m2.BF16, res_dtype=m2.F32, flags=0)
    s.update(kw)
    return L.AddNormShape(**s)


def _proj(**kw):
    s = dict(tokens=4, inputs=32, outputs=8, dtype=m2.BF16, flags=0)
    s.update(kw)
    return L.Proj8Shape(**s)


def _longs(*v):
    return (ctypes.c_int64 * len(v))(*v)


def test_add_norm_refusals(lib):
    ok = [P, P, P, P, None, P, None]      # x, residual, w, y, scales, total, stream
    for bad in (dict(batch=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(flags=2), dict(dtype=3), dict(res_dtype=7)):
        assert _call(lib, "add_norm_fwd", _norm(**bad), None, *ok) == m2.ERR_INVALID_ARG
    for bad in (dict(channels=1 << 25), dict(seqlen=1 << 31), dict(dtype=m2.F32, res_dtype=m2.BF16)):
        assert _call(lib, "add_norm_fwd", _norm(**bad), None, *ok) == m2.ERR_UNSUPPORTED
    for k in (0, 3, 5):
        assert _call(lib, "add_norm_fwd", _norm(), None, *ok[:k], None, *ok[k + 1:]) == m2.ERR_INVALID_ARG
    assert _call(lib, "add_norm_fwd", None, None, *ok) == m2.ERR_INVALID_ARG
    assert _call(lib, "add_norm_fwd", _norm(), None, *ok[:4], P, P, None) == m2.ERR_INVALID_ARG       # scales without the flag
    assert _call(lib, "add_norm_fwd", _norm(flags=1), None, *ok) == m2.ERR_INVALID_ARG               # the flag without scales
    q = [P, P, P, P, P, P, None]
    assert _call(lib, "add_norm_fwd", _norm(flags=1), None, *q[:3], P + 8, *q[4:]) == m2.ERR_INVALID_ARG   # rows of q
    st = _longs(128, 32, 128, 32, 4 * 40, 40, 128, 32)
    assert _call(lib, "add_norm_fwd", _norm(flags=1), st, *q) == m2.ERR_INVALID_ARG
    st = _longs(128, 32, 128, 32, 128, 32, 64, 32)      # total's sequences would overlap
    assert _call(lib, "add_norm_fwd", _norm(), st, *ok) == m2.ERR_INVALID_ARG
    back = [P, P, P, P, P, P, P]          # total, w, dy, dtotal, dx, dresidual, dw
    assert _call(lib, "add_norm_bwd", _norm(), None, *back, *NO_SPACE) == m2.ERR_WORKSPACE
    for k in (0, 2, 4):
        assert _call(lib, "add_norm_bwd", _norm(), None, *back[:k], None, *back[k + 1:], *SIZE) == m2.ERR_INVALID_ARG
    assert m2.add_norm_bwd_workspace_size(_norm(batch=0)) == 0 and m2.add_norm_bwd_workspace_size(_norm()) > 0


def test_quant8_refusals(lib):
    ok = dict(batch=2, seqlen=4, channels=32, dtype=m2.BF16, flags=0)
    for bad in (dict(batch=-1), dict(dtype=9), dict(flags=2), dict(flags=1)):     # blocks of one matrix only
        assert _call(lib, "quant8", _Quant8Shape(**{**ok, **bad}), None, P, P, P, None) == m2.ERR_INVALID_ARG
    assert _call(lib, "quant8", _Quant8Shape(**{**ok, "channels": 1 << 25}), None, P, P, P, None) == m2.ERR_UNSUPPORTED
    assert _call(lib, "quant8", None, None, P, P, P, None) == m2.ERR_INVALID_ARG
    for args in ((None, P, P), (P, None, P), (P, P, None), (P + 1, P, P), (P, P + 4, P)):
        assert _call(lib, "quant8", _Quant8Shape(**ok), None, *args, None) == m2.ERR_INVALID_ARG
    for st in (_longs(128, 32, 128, 24), _longs(128, 32, 64, 32), _longs(-1, 32, 128, 32)):
        assert _call(lib, "quant8", _Quant8Shape(**ok), st, P, P, P, None) == m2.ERR_INVALID_ARG


def test_proj8_refusals(lib):
    ok = [P, P, P, P, P, None]            # x, scales, w, scales, y, stream
    for bad in (dict(tokens=-1), dict(outputs=-1), dict(inputs=-1), dict(dtype=4), dict(flags=1)):
        assert _call(lib, "proj8_fwd", _proj(**bad), None, *ok) == m2.ERR_INVALID_ARG
    for bad in (dict(inputs=0), dict(tokens=(1 << 30) + 1), dict(outputs=(1 << 30) + 1)):
        assert _call(lib, "proj8_fwd", _proj(**bad), None, *ok) == m2.ERR_UNSUPPORTED
    assert _call(lib, "proj8_fwd", None, None, *ok) == m2.ERR_INVALID_ARG
    for k in range(5):
        assert _call(lib, "proj8_fwd", _proj(), None, *ok[:k], None, *ok[k + 1:]) == m2.ERR_INVALID_ARG
    for k in (0, 2):
        assert _call(lib, "proj8_fwd", _proj(), None, *ok[:k], P + 8, *ok[k + 1:]) == m2.ERR_INVALID_ARG
    for p in (_longs(24, 32, 8), _longs(40, 32, 8), _longs(32, 40, 8), _longs(32, 32, 7), _longs(0, 32, 8)):
        assert _call(lib, "proj8_fwd", _proj(), p, *ok) == m2.ERR_INVALID_ARG
    back = [P] * 7                        # dy, x, scales, w, scales, dx, dw
    assert _call(lib, "proj8_bwd", _proj(), None, *back, *NO_SPACE) == m2.ERR_WORKSPACE
    assert _call(lib, "proj8_bwd", _proj(), None, *back, P + 128, 1 << 40, None) == m2.ERR_WORKSPACE
    for k in range(5):
        assert _call(lib, "proj8_bwd", _proj(), None, *back[:k], None, *back[k + 1:], *SIZE) == m2.ERR_INVALID_ARG
    assert m2.proj8_bwd_workspace_size(_proj(tokens=0)) == 0 and m2.proj8_bwd_workspace_size(_proj(flags=2)) == 0


def test_exports_and_python_refusals(lib):
    for n in L.SYMBOLS:
        assert hasattr(lib, n)
    x = torch.zeros(2, 32)
    with pytest.raises(ValueError, match="no CPU path"):
        m2.quant8(x)
    with pytest.raises(ValueError, match="no CPU path"):
        m2.add_norm_fwd(x)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        m2.add_norm_fwd(x.half())
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        m2.proj8_fwd(x, None, None, None)
    with pytest.raises(ValueError, match="group"):
        m2.quant8(x, group="column")
    with pytest.raises(TypeError, match="dtype"):
        m2.proj8_fwd(x.to(torch.float8_e4m3fn), None, None, None, dtype=torch.float16)
    with pytest.raises(TypeError, match="torch.Tensor"):
        m2.proj8_bwd(None, None, None, None, None)
