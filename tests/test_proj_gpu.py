"""Projection operators on the GPU against plain fp64 implementations.

Bounds, from the arithmetic.  Quantising multiplies by a power of two and rounds once: results
are equal.  Norms: as for the layer's (chains of a few hundred fp32 operations, a random walk of
relative errors of 2^-24 each, below 3e-6 of the result's scale; held to 2e-5), bf16 results one
rounding more, at most 2^-8.  A norm in 8 bits: half a step of e4m3 (2^-4 of a normal value,
2^-10 scales of a subnormal one) around a value that is 2e-6 off.  Products: each of the K / 32
steps of a sum in the tensor cores is off by at most 2^-23 of the sum of magnitudes, and the
joining of a step's 32 products and of split sums by a few such errors more, counted as 8."""
import math

import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
import proj_ref as R

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


def f64(v):
    return v.detach().cpu().double() if v is not None else None


def same(got, want, what):
    """Equal values; NaN where NaN is wanted."""
    g, w = f64(got), want.reshape(got.shape)
    ok = (g == w) | (g.isnan() & w.isnan())
    assert ok.all(), f"{what}: {int((~ok).sum())} of {g.numel()} differ, first {g[~ok][:3]} for {w[~ok][:3]}"


def close(got, want, what, size=None):
    """size: the magnitudes whose relative errors reach the result (its own, where it is no sum of
    terms that cancel)."""
    g, w = f64(got), want
    assert g.shape == w.shape, what
    if not w.numel():
        return
    size = w.abs() if size is None else size
    bound = 2e-5 * (size + size.square().mean().sqrt()) + (2 ** -8 * w.abs() if got.dtype == BF16 else 0) + 1e-30
    bad = ~((g - w).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((g - w).abs() / bound).max():.3g} bounds"


class Gen:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def randn(self, *shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(dtype)

    def spread(self, *shape, dtype=F32):
        """Values over many orders of magnitude, rows of zeros among them."""
        v = torch.randn(*shape, generator=self.g) * torch.exp(4 * torch.randn(*shape[:-1], 1, generator=self.g))
        v *= torch.exp(2 * torch.randn(shape[-1], generator=self.g))
        v[..., ::7] *= torch.randn(shape[-1], generator=self.g)[::7].abs() < 1.5
        return v.to(dtype)


def pitched(v, pad, lead=0, fill=NAN):
    """The same values as a column slice of a wider tensor on the GPU."""
    wide = torch.full((*v.shape[:-1], v.shape[-1] + pad + lead), fill, dtype=torch.float32).to(v.dtype).cuda()
    out = wide[..., lead:lead + v.shape[-1]]
    out.copy_(v)
    return out


# ---- quant8 -------------------------------------------------------------------------------------

QUANT = [  # shape, dtype, group, pad, lead
    ((1, 1), F32, "row", 0, 0),
    ((1, 1), BF16, "block", 0, 0),
    ((1, 128), BF16, "row", 0, 0),
    ((3, 129), F32, "row", 0, 0),
    ((130, 127), BF16, "row", 3, 1),
    ((2, 5, 272), BF16, "row", 0, 0),
    ((2, 3, 257), F32, "row", 1, 0),
    ((7, 1, 64), BF16, "row", 8, 8),
    ((129, 640), F32, "row", 4, 4),
    ((1, 4104), BF16, "row", 0, 0),
    ((128, 128), F32, "block", 0, 0),
    ((129, 257), F32, "block", 0, 0),
    ((300, 136), BF16, "block", 8, 0),
    ((127, 255), BF16, "block", 1, 1),
]


@pytest.mark.parametrize("case", QUANT, ids=str)
def test_quant8(case):
    shape, dt, group, pad, lead = case
    x = Gen(1).spread(*shape, dtype=dt)
    rows, cols = (1, 128) if group == "row" else (128, 128)
    want = R.quant(f64(x).flatten(0, -2), rows, cols)
    q, s = m2.quant8(pitched(x, pad, lead), group=group)
    assert q.shape == x.shape and q.dtype == E4M3 and s.dtype == torch.float8_e8m0fnu
    assert q.stride(-2) % 16 == 0 and q.data_ptr() % 16 == 0
    same(s, want[1], "scales")
    same(q, want[0], "q")


def test_quant8_edges():
    """The largest values of each scale, ties, subnormals of both types, infinities and NaN."""
    x = torch.zeros(12, 256)
    x[0] = 448.0
    x[1, 0], x[1, 1:] = 448.0, torch.arange(255) / 16
    x[2, 0] = math.nextafter(448.0, 1e9) + 3e-5
    x[3, :128] = 2.0 ** -149
    x[4, :] = 1e38 * torch.linspace(-3.4, 3.4, 256)
    x[5, 3], x[5, 4], x[5, 5] = INF, -INF, 1.0
    x[6, 7], x[6, 200] = NAN, -3.0
    x[7, :128] = INF
    x[8] = 2.0 ** -127 * torch.linspace(-448, 448, 256)
    x[9] = -0.0
    x[10, :] = torch.linspace(-1, 1, 256) * 2.0 ** -140
    x[11] = 1.75 * 2.0 ** 100
    for dt in (F32, BF16):
        v = x.to(dt)
        for group, r, c in (("row", 1, 128), ("block", 128, 128)):
            q, s = m2.quant8(v.cuda(), group=group)
            want = R.quant(f64(v), r, c)
            same(s, want[1], f"{group} scales")
            same(q, want[0], f"{group} q")


def test_quant8_given_outputs_and_neighbours():
    """Outputs inside a larger buffer: nothing beside them is touched."""
    x = Gen(2).randn(5, 3, 130)
    room = torch.full((5, 4, 160), 77, dtype=torch.uint8, device="cuda")
    q = room.view(E4M3)[:, :3, 16:146]
    s = torch.empty(5, 3, 2, dtype=torch.float8_e8m0fnu, device="cuda")
    got = m2.quant8(x.cuda(), q=q, scales=s)
    assert got[0] is q and got[1] is s
    want = R.quant(f64(x).flatten(0, 1), 1, 128)
    same(q, want[0], "q")
    same(s, want[1], "scales")
    keep = room.clone()
    keep[:, :3, 16:146] = 77
    assert (keep == 77).all()


# ---- add_norm -----------------------------------------------------------------------------------

NORM = [  # shape, dtype, residual's dtype (None: no residual), w, pad, lead
    ((1, 1, 1), F32, F32, True, 0, 0),
    ((2, 3, 64), BF16, F32, True, 0, 0),
    ((2, 3, 65), BF16, F32, True, 0, 0),
    ((3, 1, 128), BF16, BF16, False, 0, 0),
    ((11, 100), F32, F32, True, 4, 4),
    ((11, 256), BF16, F32, True, 8, 0),
    ((2, 5, 513), BF16, BF16, True, 1, 1),
    ((2, 9, 1000), F32, F32, True, 0, 0),
    ((2, 9, 1001), F32, F32, False, 0, 0),
    ((3, 2560), BF16, F32, True, 0, 0),
    ((1, 2, 5120), BF16, BF16, True, 0, 0),
    ((2, 8200), BF16, F32, True, 0, 0),
    ((2, 8196), F32, F32, True, 0, 0),
    ((2, 8193), F32, F32, True, 0, 0),
    ((2, 20000), BF16, F32, True, 0, 0),
    ((2, 20001), BF16, BF16, True, 0, 0),
    ((2, 4, 96), BF16, None, True, 0, 0),
    ((2, 4, 97), F32, None, False, 3, 0),
]


def _norm_inputs(case, seed=3):
    shape, dt, rt, with_w, pad, lead = case
    r = Gen(seed)
    x = r.spread(*shape, dtype=dt)
    res = r.spread(*shape, dtype=rt) if rt is not None else None
    w = 1 + r.randn(shape[-1], scale=0.3) if with_w else None
    total = (x.float() + res.float()).to(rt) if res is not None else x
    cu = lambda v: pitched(v, pad, lead) if v is not None else None          # noqa: E731
    return x, res, w, total, cu


@pytest.mark.parametrize("case", NORM, ids=str)
def test_add_norm_fwd(case):
    x, res, w, total, cu = _norm_inputs(case)
    y, t = m2.add_norm_fwd(cu(x), cu(res), w.cuda() if w is not None else None, eps=1e-4)
    assert y.dtype == x.dtype and t.dtype == total.dtype
    same(t, f64(total), "total")
    want = R.add_norm(f64(total), f64(w), 1e-4)
    g = f64(y)
    # rows are of many sizes: a row's own scale
    scale = want.abs() + want.square().mean(-1, keepdim=True).sqrt()
    bound = 2e-5 * scale + (2 ** -8 * want.abs() if y.dtype == BF16 else 0) + 1e-30
    assert ((g - want).abs() <= bound).all()


@pytest.mark.parametrize("case", NORM, ids=str)
def test_add_norm_fwd_quant(case):
    x, res, w, total, cu = _norm_inputs(case)
    q, s, t = m2.add_norm_fwd(cu(x), cu(res), w.cuda() if w is not None else None, eps=1e-4, quant=True)
    D = x.shape[-1]
    assert q.dtype == E4M3 and q.shape == x.shape and s.shape == (*x.shape[:-1], -(-D // 128))
    same(t, f64(total), "total")
    want = R.add_norm(f64(total), f64(w), 1e-4)
    wide = f64(s).repeat_interleave(128, -1)[..., :D]
    # the scale is right for a largest value that is 2e-6 off
    for j in range(s.shape[-1]):
        top = want[..., 128 * j:128 * j + 128].abs().amax(-1).flatten().tolist()
        for v, got in zip(top, f64(s)[..., j].flatten().tolist()):
            assert got in {2.0 ** R.scale_exponent(v * f) for f in (1 - 2e-6, 1 + 2e-6)}
    bound = torch.maximum(2 ** -4 * want.abs(), 2 ** -10 * wide) + 2e-6 * want.abs() + 1e-35
    assert ((f64(q) * wide - want).abs() <= bound).all()


@pytest.mark.parametrize("with_dt", [True, False])
@pytest.mark.parametrize("case", [c for c in NORM if c[2] is not None], ids=str)
def test_add_norm_bwd(case, with_dt):
    x, res, w, total, cu = _norm_inputs(case, 4)
    r = Gen(5)
    total = r.randn(*x.shape, dtype=total.dtype)
    dy, dt = r.randn(*x.shape, dtype=x.dtype), r.randn(*x.shape, dtype=total.dtype) if with_dt else None
    g = m2.add_norm_bwd(cu(total), w.cuda() if w is not None else None, cu(dy), cu(dt), eps=1e-4)
    dx, dw = R.add_norm_bwd(f64(total), f64(w), 1e-4, f64(dy), f64(dt))
    assert g["dx"].dtype == x.dtype and g["dresidual"].dtype == total.dtype
    assert (g["dresidual"] is g["dx"]) == (x.dtype == total.dtype)
    # dx = r g - r n mean(g n) + dtotal: each term has relative errors of fp32 operations of its own,
    # and the first two cancel to eps / (t^2 + eps) of their size in a row of one channel
    size = R.add_norm_bwd_size(f64(total), f64(w), 1e-4, f64(dy), f64(dt))
    close(g["dx"], dx, "dx", size)
    close(g["dresidual"], dx, "dresidual", size)
    if w is None:
        assert g["dw"] is None
    else:
        close(g["dw"], dw, "dw")


def test_add_norm_bwd_many_tokens():
    """More tokens than teams, so that a team takes several, at widths of each kind of team."""
    for D, dt in ((40, BF16), (500, BF16), (1031, F32), (20000, BF16)):
        r = Gen(D)
        n = 12000 if D < 100 else 3000 if D < 2000 else 700
        total, dy, dt_ = r.randn(n, D), r.randn(n, D, dtype=dt), r.randn(n, D)
        w = 1 + r.randn(D, scale=0.3)
        g = m2.add_norm_bwd(total.cuda(), w.cuda(), dy.cuda(), dt_.cuda())
        dx, dw = R.add_norm_bwd(f64(total), f64(w), 1e-5, f64(dy), f64(dt_))
        close(g["dx"], dx, "dx")
        close(g["dresidual"], dx, "dresidual")
        close(g["dw"], dw, "dw")


def test_add_norm_of_nothing():
    for shape in ((0, 4, 32), (2, 0, 32), (0, 32)):
        x = torch.zeros(shape, device="cuda")
        y, t = m2.add_norm_fwd(x, x)
        assert y.shape == t.shape == x.shape
        q, s, t = m2.add_norm_fwd(x, x, quant=True)
        assert q.shape == x.shape and s.shape == (*shape[:-1], 1)
        g = m2.add_norm_bwd(x, torch.ones(32, device="cuda"), x)
        assert (g["dw"] == 0).all() and g["dx"].shape == x.shape
        assert m2.quant8(x)[0].shape == x.shape


def test_add_norm_begins_a_residual_in_f32():
    x = Gen(6).randn(3, 70, dtype=BF16)
    y, t = m2.add_norm_fwd(x.cuda(), residual_f32=True)
    assert t.dtype == F32 and y.dtype == BF16
    same(t, f64(x), "total")
    close(y, R.add_norm(f64(x), None, 1e-5), "y")


# ---- proj8 --------------------------------------------------------------------------------------

PROJ = [  # M, K, N
    (1, 1, 1),
    (1, 128, 128),
    (3, 130, 5),
    (17, 64, 129),
    (1, 1095, 300),
    (16, 512, 200),
    (33, 700, 257),
    (64, 2560, 64),
    (128, 128, 128),
    (129, 640, 130),
    (200, 1000, 333),
    (257, 513, 512),
    (2, 4096, 1031),
    (520, 96, 70),
]


def _operands(M, K, N, seed=7):
    """(x, w) quantised on the GPU and as the fp64 values that they stand for."""
    r = Gen(seed)
    x, w = r.randn(M, K) * torch.exp(r.randn(M, 1)), r.randn(N, K, scale=K ** -0.5) * torch.exp(r.randn(N, 1))
    x[:, ::9] *= 20
    qx, qw = m2.quant8(x.cuda()), m2.quant8(w.cuda(), group="block")
    vx, vw = R.dequant(f64(qx[0]), f64(qx[1]), 1, 128), R.dequant(f64(qw[0]), f64(qw[1]), 128, 128)
    return (*qx, *qw), vx, vw


def product(got, a, b, what):
    """got = a b for fp64 a, b."""
    want, size = a @ b, a.abs() @ b.abs()
    steps = -(-a.shape[1] // 32) + 8
    bound = steps * 2.0 ** -23 * size + (2 ** -8 * want.abs() if got.dtype == BF16 else 0) + 1e-37
    bad = ~((f64(got) - want).abs() <= bound)
    # a sum behind fp32's largest value is an infinity (the type's range, not a rounding)
    bad &= ~((want.abs() > torch.finfo(F32).max) & (f64(got) == INF * want.sign()))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((f64(got) - want).abs() / bound).max():.3g} bounds"


@pytest.mark.parametrize("dt", [F32, BF16], ids=("f32", "bf16"))
@pytest.mark.parametrize("case", PROJ, ids=str)
def test_proj8_fwd(case, dt):
    M, K, N = case
    ops, x, w = _operands(M, K, N)
    y = m2.proj8_fwd(*ops, dtype=dt)
    assert y.shape == (M, N) and y.dtype == dt
    product(y, x, w.t(), "y")
    assert torch.equal(y, m2.proj8_fwd(*ops, dtype=dt))
    assert m2.device_error() == 0


@pytest.mark.parametrize("dt", [F32, BF16], ids=("f32", "bf16"))
@pytest.mark.parametrize("case", PROJ, ids=str)
def test_proj8_bwd(case, dt):
    M, K, N = case
    ops, x, w = _operands(M, K, N)
    r = Gen(8)
    dy = (r.randn(M, N) * torch.exp(2 * r.randn(M, 1)) * 1e-3).to(dt)
    g = m2.proj8_bwd(dy.cuda(), *ops)
    assert g["dx"].shape == (M, K) and g["dx"].dtype == dt and g["dw"].shape == (N, K) and g["dw"].dtype == F32
    d = f64(dy)
    product(g["dx"], R.dequant(*R.quant(d, 1, 128), 1, 128), w, "dx")
    product(g["dw"], R.dequant(*R.quant(d, 128, 1), 128, 1).t(), R.dequant(*R.quant(x, 128, 1), 128, 1), "dw")
    again = m2.proj8_bwd(dy.cuda(), *ops, need_dx=False)
    assert again["dx"] is None and torch.equal(again["dw"], g["dw"])
    again = m2.proj8_bwd(dy.cuda(), *ops, need_dw=False)
    assert again["dw"] is None and torch.equal(again["dx"], g["dx"])
    assert m2.device_error() == 0


def test_proj8_gradients_are_near_the_product_s():
    """dx and dw against those of the unrounded product: a rounding to e4m3 is at most 2^-4 of a
    value, one operand's in dx, two operands' in dw, of independent sign: below 2^-4 and 2^-3 of
    the result's norm."""
    ops, x, w = _operands(300, 400, 260)
    dy = Gen(9).randn(300, 260)
    g = m2.proj8_bwd(dy.cuda(), *ops)
    for got, want, most in ((g["dx"], f64(dy) @ w, 2 ** -4), (g["dw"], f64(dy).t() @ x, 2 ** -3)):
        assert (f64(got) - want).norm() <= most * want.norm()


@pytest.mark.parametrize("M", [1, 3, 150])
def test_proj8_slices(M):
    """Operands, result and gradient as slices of wider buffers; three dimensions; nothing beside
    the result is written."""
    K, N, b = 200, 90, 2
    r = Gen(10)
    x, w = r.randn(b, M, K), r.randn(N, K)
    wide = torch.empty(b, M, 240, dtype=E4M3, device="cuda")
    wide.view(torch.uint8).fill_(0x7f)                       # NaN
    q, s = m2.quant8(x.cuda(), q=wide[..., 16:216])
    ww = torch.empty(N, 224, dtype=E4M3, device="cuda")
    ww.view(torch.uint8).fill_(0x7f)
    qw, sw = m2.quant8(w.cuda(), group="block", q=ww[:, :K])
    vx = R.dequant(f64(q).flatten(0, 1), f64(s).flatten(0, 1), 1, 128)
    vw = R.dequant(f64(qw), f64(sw), 128, 128)
    room = torch.full((b, M, 97), 7.0, device="cuda")
    y = m2.proj8_fwd(q, s, qw, sw, y=room[..., 5:5 + N])
    product(y.flatten(0, 1).contiguous(), vx, vw.t(), "y")
    assert (room[..., :5] == 7).all() and (room[..., 5 + N:] == 7).all()
    dy = pitched(r.randn(b, M, N, dtype=BF16), 3, 2)
    g = m2.proj8_bwd(dy, q, s, qw, sw)
    assert g["dx"].shape == x.shape
    dx, dw = R.proj_bwd(f64(dy).flatten(0, 1), vx, vw)
    close(g["dx"].flatten(0, 1), dx, "dx")
    close(g["dw"], dw, "dw")


def test_proj8_of_nothing():
    (q, s, wq, ws), _, _ = _operands(4, 32, 8)
    assert m2.proj8_fwd(q[:0], s[:0], wq, ws).shape == (0, 8)
    g = m2.proj8_bwd(torch.zeros(0, 8, device="cuda"), q[:0], s[:0], wq, ws)
    assert g["dx"].shape == (0, 32) and (g["dw"] == 0).all()
    g = m2.proj8_bwd(torch.zeros(4, 0, device="cuda"), q, s, wq[:0], ws[:0])
    assert (g["dx"] == 0).all() and g["dw"].shape == (0, 32)


def test_proj8_nan_stays_in_its_row():
    x = Gen(11).randn(70, 300)
    x[3, 7], x[60, 299] = NAN, INF
    w = Gen(12).randn(140, 300)
    q, s = m2.quant8(x.cuda())
    y = m2.proj8_fwd(q, s, *m2.quant8(w.cuda(), group="block"))
    bad = y.isnan().any(1).cpu()
    assert bad.nonzero().flatten().tolist() == [3, 60] and y[3].isnan().all() and y[60].isnan().all()


def test_proj8_wide_scales():
    """Scales at both ends of their range: 2^-127 with 2^120 and back."""
    K = 256
    x = torch.zeros(5, K)
    x[0, :128], x[0, 128:] = 2.0 ** -140, 1.0
    x[1, :] = 2.0 ** 127
    x[2, 5] = 2.0 ** -149
    x[3, :] = -2.0 ** 100
    w = torch.ones(130, K) * 2.0 ** -100
    w[:, :128] = 3.0
    (q, s), (wq, ws) = m2.quant8(x.cuda()), m2.quant8(w.cuda(), group="block")
    y = m2.proj8_fwd(q, s, wq, ws, dtype=F32)
    product(y, R.dequant(f64(q), f64(s), 1, 128), R.dequant(f64(wq), f64(ws), 128, 128).t(), "y")


# ---- together -----------------------------------------------------------------------------------

def _chain(x, res, wn, w, dout):
    """norm -> projection, forward and backward, as a layer runs them."""
    q, s, total = m2.add_norm_fwd(x, res, wn, quant=True)
    wq, ws = m2.quant8(w, group="block")
    y = m2.proj8_fwd(q, s, wq, ws)
    g = m2.proj8_bwd(dout, q, s, wq, ws)
    n = m2.add_norm_bwd(total, wn, g["dx"], None)
    return y, g["dw"], n["dx"], n["dresidual"], n["dw"]


def test_chain_against_the_unrounded_layer():
    """The norm, the projection and their gradients as a layer runs them, against fp64 autograd of
    the layer without 8 bits.  Roundings to e4m3 are at most 2^-4 of a value and independent, so
    that a result's norm moves by less than 2^-4 for each rounded operand: two in y, two in dx (dy
    and w), three in dw (dy, and x twice)."""
    r = Gen(13)
    x, res, wn = r.randn(2, 90, 384, dtype=BF16), r.randn(2, 90, 384), 1 + r.randn(384, scale=0.2)
    w, dout = r.randn(520, 384, scale=384 ** -0.5), r.randn(2, 90, 520, dtype=BF16)
    y, dw, dx, dres, dwn = _chain(*(v.cuda() for v in (x, res, wn, w, dout)))
    v = [f64(t).requires_grad_() for t in (x, wn, w)]
    total = v[0] + f64(res)
    ref = total / (total.square().mean(-1, keepdim=True) + 1e-5).sqrt() * v[1] @ v[2].t()
    gx, gwn, gw = torch.autograd.grad(ref, v, f64(dout))
    for got, want, n in ((y, ref.detach(), 2), (dw, gw, 3), (dx, gx, 2), (dres, gx, 2), (dwn, gwn, 2)):
        assert (f64(got) - want).norm() <= n * 2 ** -4 * want.norm()


def test_chain_captured_and_on_another_stream():
    """The same bits from a captured graph replayed on new inputs, and on a stream of the caller's."""
    r = Gen(14)
    sets = [tuple(v.cuda() for v in (r.randn(3, 50, 264, dtype=BF16), r.randn(3, 50, 264), 1 + r.randn(264, scale=0.2),
                                     r.randn(200, 264), r.randn(3, 50, 200, dtype=BF16))) for _ in range(2)]
    want = [_chain(*s) for s in sets]
    held = tuple(t.clone() for t in sets[0])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = _chain(*held)
    for s, w in zip(sets, want):
        for h, t in zip(held, s):
            h.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    x, res, wn, w, dout = sets[1]
    q, s, total = m2.add_norm_fwd(x, res, wn, quant=True, stream=st)
    wq, ws = m2.quant8(w, group="block", stream=st)
    y = m2.proj8_fwd(q, s, wq, ws, stream=st)
    gr = m2.proj8_bwd(dout, q, s, wq, ws, stream=st)
    n = m2.add_norm_bwd(total, wn, gr["dx"], None, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, gr["dw"], n["dx"], n["dresidual"], n["dw"]), want[1]))


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, do not disturb each other."""
    (a, _, _), (b, _, _) = _operands(700, 640, 520, 15), _operands(300, 900, 1000, 16)
    da, db = Gen(17).randn(700, 520).cuda(), Gen(18).randn(300, 1000).cuda()
    wa, wb = m2.proj8_bwd(da, *a), m2.proj8_bwd(db, *b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append((m2.proj8_bwd(da, *a, stream=s), m2.proj8_bwd(db, *b, stream=t)))
    torch.cuda.synchronize()
    for ga, gb in got:
        for k in ("dx", "dw"):
            assert torch.equal(ga[k], wa[k]) and torch.equal(gb[k], wb[k])


# ---- refusals -----------------------------------------------------------------------------------

def test_refusals():
    (q, s, wq, ws), _, _ = _operands(6, 200, 40)
    x = torch.zeros(2, 3, 64, device="cuda")
    with pytest.raises(ValueError, match="16-byte"):
        m2.proj8_fwd(q.contiguous(), s, wq, ws)
    with pytest.raises(ValueError, match="16-byte"):
        m2.quant8(x, q=torch.empty(2, 3, 72, dtype=E4M3, device="cuda")[..., :64])
    with pytest.raises(TypeError, match="e8m0"):
        m2.proj8_fwd(q, s.view(torch.uint8), wq, ws)
    with pytest.raises(ValueError, match="x_scales must have shape"):
        m2.proj8_fwd(q, s[:, :1].contiguous(), wq, ws)
    with pytest.raises(ValueError, match="w_scales must have shape"):
        m2.proj8_fwd(q, s, wq, ws.t().contiguous())
    with pytest.raises(ValueError, match="w must have shape"):
        m2.proj8_fwd(q, s, wq[:, :190], ws)
    with pytest.raises(ValueError, match="even distances"):
        wide, _ = m2.quant8(torch.zeros(2, 4, 64, device="cuda"))
        m2.proj8_fwd(wide[:, :3], torch.zeros(2, 3, 1, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu),
                     *m2.quant8(torch.zeros(8, 64, device="cuda"), group="block"))
    with pytest.raises(ValueError, match="dy must have shape"):
        m2.proj8_bwd(torch.zeros(6, 41, device="cuda"), q, s, wq, ws)
    with pytest.raises(ValueError, match="must not overlap"):
        m2.proj8_bwd(torch.zeros(6, 40, device="cuda"), q, s, wq, ws, workspace=q.new_empty(0).set_(q.untyped_storage()))
    with pytest.raises(m2.Mamba2Error):
        m2.proj8_bwd(torch.zeros(6, 40, device="cuda"), q, s, wq, ws, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="2 dimensions"):
        m2.quant8(x, group="block")
    with pytest.raises(TypeError, match="residual"):
        m2.add_norm_fwd(x, x.bfloat16())
    with pytest.raises(ValueError, match="must not overlap"):
        m2.add_norm_fwd(x, x.clone(), total=x)
    with pytest.raises(ValueError, match="quant only"):
        m2.add_norm_fwd(x, scales=torch.zeros(2, 3, 1, device="cuda"))
    with pytest.raises(ValueError, match="w must have shape"):
        m2.add_norm_fwd(x, None, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        m2.add_norm_fwd(x.transpose(1, 2))
    with pytest.raises(ValueError, match="total is required"):
        m2.add_norm_bwd(None, None, x)
    with pytest.raises(ValueError, match="2 or 3 dimensions"):
        m2.quant8(torch.zeros(4, device="cuda"))
