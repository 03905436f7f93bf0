"""Layer operators at sizes that take the code the layer's own sizes take: the
convolution's rings refilled many times, the norm's backward teams with more than one
token each, the scan's backward with four channels a lane in turn.  Each test asserts that
its case does select that code, from the workspace the call asks for.

Bounds as in test_layer_gpu.  The longest sums here are the convolution's dw over 16000
tokens and the scan's dA and ddt_bias over 2000: a thread adds at most a few hundred terms
one after another before the parts are joined, so their rounding stays a random walk of a
few hundred steps of 2^-24 against a sum whose scale is its own rms."""
import ctypes

import pytest
import torch

import layer_ref as R
import mamba_ssd_chunked_02_gb300 as m2
from mamba_ssd_chunked_02_gb300 import layer as L
from test_layer_gpu import BF16, F32, ORDER, Gen, cu, f64, lens, pitched, scan_inputs, spoil

pytestmark = pytest.mark.gpu


def close(got, want, what):
    """test_layer_gpu.close where `want` is."""
    assert got is not None and tuple(got.shape) == tuple(want.shape), what
    g, w = got.detach().to(want.device).double(), want.double()
    bound = 2e-5 * (w.abs() + w.square().mean().sqrt()) + (2 ** -8 * w.abs() if got.dtype == BF16 else 0) + 1e-30
    bad = ~((g - w).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((g - w).abs() / bound).max():.3g} bounds"


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


def code(dtype):
    return m2.BF16 if dtype == BF16 else m2.F32


def slots(name, shape, row):
    """Partial sums of `row` floats that a backward's workspace holds."""
    return L._fn(name)(ctypes.addressof(shape)) // (4 * row)


# ---- conv ---------------------------------------------------------------------------------------

CONV = [  # b, T, D, W, dtype, act, bias, init, ragged, pad, lead
    (8, 2000, 2052, 4, BF16, True, True, True, True, 0, 0),      # four channels a thread
    (8, 2000, 2050, 4, BF16, True, True, False, False, 2, 2),    # two
    (5, 2003, 2051, 3, BF16, True, True, True, True, 1, 1),      # one: no ring
    (8, 1501, 2052, 4, F32, True, False, True, True, 4, 4),
    (6, 1500, 1027, 2, F32, False, True, True, True, 1, 1),
]


def conv_wide(x, w, bias, init, lengths, act, dy=None, dfinal=None):
    """layer_ref.conv with all tokens at once."""
    b, T, D = x.shape
    W = w.shape[1]
    ends = torch.full((b,), T, device=x.device) if lengths is None else lengths.long().clamp(0, T)
    real = (torch.arange(T, device=x.device)[None] < ends[:, None])[..., None]
    x = torch.where(real, x, torch.zeros_like(x))
    seen = torch.cat([init if init is not None else x.new_zeros(b, W - 1, D), x], 1)
    s = sum(seen[:, k:k + T] * w[:, k] for k in range(W))
    if bias is not None:
        s = s + bias
    y, slope = R.silu(s) if act else (s, torch.ones_like(s))
    last = torch.arange(b, device=x.device)[:, None], ends[:, None] + torch.arange(W - 1, device=x.device)
    if dy is None:
        return torch.where(real, y, torch.zeros_like(y)), seen[last]
    ds = torch.where(real, dy, torch.zeros_like(dy)) * slope
    dseen = torch.zeros_like(seen)
    for k in range(W):
        dseen[:, k:k + T] += ds * w[:, k]
    if dfinal is not None:
        dseen[last] += dfinal
    return dict(dx=torch.where(real, dseen[:, W - 1:], torch.zeros_like(x)), dinit=dseen[:, :W - 1],
                dw=torch.stack([(ds * seen[:, k:k + T]).sum((0, 1)) for k in range(W)], 1), dbias=ds.sum((0, 1)))


def test_conv_wide_is_the_token_by_token_form():
    r = Gen(40)
    x, w, bias, init = r.randn(4, 7, 3).double(), r.randn(3, 4).double(), r.randn(3).double(), r.randn(4, 3, 3).double()
    dy, df, n = r.randn(4, 7, 3).double(), r.randn(4, 3, 3).double(), torch.tensor([7, 0, 2, 5])
    for a, b in zip(conv_wide(x, w, bias, init, n, True), R.conv(x, w, bias, init, n)):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)
    a, b = conv_wide(x, w, bias, init, n, True, dy, df), R.conv(x, w, bias, init, n, True, dy, df)
    assert all(torch.allclose(a[k], b[k], rtol=1e-12, atol=1e-12) for k in b)


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(case):
    b, T, D, W, dt, act, with_bias, with_init, ragged, pad, lead = case
    # Stretches of 32 tokens and more (the backward's stretch, from its slots of 4 stretches
    # each): at least (32 - 3) / 4 = 7 groups pass through a ring of at most four.  The
    # forward's start is a seventh of the backward's, but with as many waves of threads the
    # same lengths are best for it too.
    assert 0 < slots("conv_bwd_ws", L.ConvShape(b, T, D, W, code(dt), 0), D * (W + 1)) <= b * -(-T // (4 * 32))
    r = Gen(41)
    x, w = r.randn(b, T, D, dtype=dt), r.randn(D, W, scale=0.5)
    bias = r.randn(D, scale=0.5) if with_bias else None
    init = r.randn(b, W - 1, D, dtype=dt) if with_init else None
    dy, df = r.randn(b, T, D, dtype=dt), r.randn(b, W - 1, D, dtype=dt)
    n = lens(ragged, b, T)
    xd, dyd = pitched(spoil(x, n), pad, lead), pitched(spoil(dy, n), pad, lead)
    ref = [f64(cu(v)) for v in (x, w, bias, init)]
    y, fin = m2.conv_fwd(xd, cu(w), cu(bias), cu(init), cu(n), silu=act)
    yr, fr = conv_wide(*ref, cu(n), act)
    close(y, yr, "y")
    assert torch.equal(fin.double(), fr)
    args = (xd, cu(w), cu(bias), cu(init), dyd, cu(df), cu(n))
    g = m2.conv_bwd(*args, silu=act)
    want = conv_wide(*ref, cu(n), act, f64(cu(dy)), f64(cu(df)))
    for k in want:
        if (k == "dbias" and bias is None) or (k == "dinit" and init is None):
            assert g[k] is None
        else:
            close(g[k], want[k], k)
    assert same(g, m2.conv_bwd(*args, silu=act))


# ---- norm ---------------------------------------------------------------------------------------

NORM = [  # b, T, D, G, dtype, gate, weight, pad
    (4, 1100, 128, 2, BF16, "first", True, 0),      # a warp a team: one vector a lane ...
    (3, 2100, 512, 1, BF16, "after", True, 8),      # two
    (3, 1700, 768, 1, BF16, "first", True, 0),      # three
    (3, 1100, 1280, 2, BF16, "first", True, 0),     # five of four channels
    (3, 2100, 300, 1, BF16, None, True, 4),
    (2, 3100, 66, 1, BF16, "first", True, 1),       # misaligned rows: one channel, not staged
    (3, 2100, 640, 1, F32, "after", True, 0),
    (4, 1600, 65, 1, F32, "first", True, 0),
    (2, 250, 5120, 1, BF16, "first", True, 0),      # a block a team
    (2, 250, 5120, 1, F32, "after", True, 0),
    (2, 250, 10240, 1, BF16, "first", True, 0),     # two vectors a thread
    (2, 250, 4100, 2, BF16, "first", True, 2),      # narrow accesses, four of them
    (2, 250, 2051, 1, BF16, "after", True, 1),
    (2, 160, 20000, 1, BF16, "first", True, 0),     # any number of vectors: read twice, dw in memory
    (2, 160, 9001, 1, BF16, "after", True, 0),
    (2, 160, 9004, 1, F32, None, True, 0),
]


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_backward_with_several_tokens_a_team(case):
    b, T, D, G, dt, gate, weight, pad = case
    sh = L.NormShape(b, T, D, G, 1e-5, code(dt), 0 if gate != "after" else m2.layer.NORM_GATE_AFTER)
    assert 0 < 2 * slots("norm_bwd_ws", sh, D) < b * T      # some teams have three
    r = Gen(42)
    x, dy = r.randn(b, T, D, dtype=dt), r.randn(b, T, D, dtype=dt)
    z = r.randn(b, T, D, dtype=dt) if gate else None
    w = 1 + r.randn(D, scale=0.1) if weight else None
    first = gate != "after"
    args = (pitched(x, pad, pad), cu(w), pitched(z, pad, pad) if gate else None, pitched(dy, pad, pad))
    g = m2.norm_bwd(*args, ngroups=G, eps=1e-5, gate_first=first)
    want = R.norm(*[f64(cu(v)) for v in (x, w, z)], G, 1e-5, first, f64(cu(dy)))
    for k in ("dx", "dz", "dw"):
        if k == "dz" and z is None:
            assert g[k] is None
        else:
            close(g[k], want[k], k)
    assert same(g, m2.norm_bwd(*args, ngroups=G, eps=1e-5, gate_first=first))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 2])
def test_norm_at_every_width(dt, pad):
    """Groups of all sizes up to 4200 in steps of 3 and of 8, and larger ones: every access width, team
    and staging room."""
    widths = sorted({*range(1, 4200, 3), *range(8, 4200, 8), *range(4224, 17000, 352)})
    r = Gen(45)
    whole = [cu(r.randn(2, 2, widths[-1] + pad, dtype=dt)) for _ in range(3)]
    w = cu(1 + r.randn(widths[-1], scale=0.1))
    for S in widths:
        x, z, dy = (v[:, :, pad:pad + S] if pad else v[:, :, :S].contiguous() for v in whole)
        y, g = m2.norm_fwd(x, w[:S], z), m2.norm_bwd(x, w[:S], z, dy)
        ref = [f64(v) for v in (x, w[:S], z)]
        close(y, R.norm(*ref, 1, 1e-5), f"y of {S}")
        want = R.norm(*ref, 1, 1e-5, True, f64(dy))
        for k in want:
            close(g[k], want[k], f"{k} of {S}")


# ---- scan ---------------------------------------------------------------------------------------

SCAN = [  # b, T, D, N, G, dtype, softplus, D, z, bias, init, ragged, pad
    (5, 331, 1000, 16, 1, BF16, True, True, True, True, True, True, 0),
    (5, 331, 999, 16, 1, F32, True, True, True, True, True, True, 0),
    (3, 325, 1300, 16, 2, F32, True, True, False, True, True, True, 2),
    (5, 430, 1027, 8, 1, BF16, True, True, True, True, True, True, 1),
    (4, 420, 1028, 8, 2, F32, True, False, True, True, True, False, 0),
    (5, 300, 515, 32, 1, F32, True, True, True, True, False, True, 0),
    (4, 300, 516, 32, 1, BF16, False, True, False, True, True, True, 0),
    (4, 300, 330, 64, 1, BF16, True, True, True, True, True, False, 4),
    (5, 260, 150, 128, 1, F32, True, True, False, True, True, True, 0),
    (4, 260, 300, 128, 2, BF16, True, True, True, True, True, False, 0),
]


def turns(b, T, D, N, G, have):
    """Channels a lane takes in turn (4 or 1) that give a scan backward workspace of `have` bytes,
    for some number of stretches: states every 8 tokens and their sums of steps; per stretch two
    states, sums and the parts of dA, dD and ddt_bias; dB and dC per block of channels."""
    def up(v):
        return (v + 255) // 256 * 256

    found = set()
    for kk in (4, 1):
        block = 128 // (N // 4) * kk
        ncb = -(-(D // G) // block)
        for seg in range(1, 65):
            nck = -(-T // 8)
            parts = [b * nck * D * N, b * nck * D, 2 * seg * b * D * N if seg > 1 else 0,
                     seg * b * D if seg > 1 else 0, ncb * b * T * G * 2 * N, seg * b * D * N, seg * b * 2 * D]
            if sum(up(4 * v) for v in parts) == have:
                found.add(kk)
    return found


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_backward_with_four_channels_in_turn(case):
    b, T, D, N, G, dt, softplus = case[:7]
    pad = case[-1]
    sh = L.ScanShape(b, T, D, N, G, code(dt), int(softplus))
    assert turns(b, T, D, N, G, m2.scan_bwd_workspace_size(sh)) == {4}
    v, n, r = scan_inputs(case, 43)
    dy, df = r.randn(b, T, D, dtype=dt), r.randn(b, D, N)
    dev = {k: cu(v[k]) for k in ORDER}
    for k in ("x", "dt", "z"):
        if v[k] is not None:
            dev[k] = pitched(spoil(v[k], n), pad, pad)
    for k in ("B", "C"):
        dev[k] = pitched(spoil(v[k], n).flatten(2), pad, pad).unflatten(2, (G, N))
    dyd = pitched(spoil(dy, n), pad, pad)
    args = [dev[k] for k in ORDER]
    g = m2.scan_bwd(*args, dyd, cu(df), cu(n), dt_softplus=softplus)
    ref = [f64(v[k]) for k in ORDER]
    want = R.scan(*ref, n, softplus, f64(dy), f64(df))
    absent = dict(dD=v["D"], dz=v["z"], ddt_bias=v["dt_bias"], dinit=v["init"])
    for k in want:
        if k in absent and absent[k] is None:
            assert g[k] is None
        else:
            close(g[k], want[k], k)
    assert same(g, m2.scan_bwd(*args, dyd, cu(df), cu(n), dt_softplus=softplus))


def test_scan_rows_in_turns_with_odd_channels():
    """Three slices and single-channel accesses: more rows than the GPU holds."""
    b, T, D, N = 40, 400, 1001, 16
    v, n, _ = scan_inputs((b, T, D, N, 1, F32, True, True, True, True, True, True, 0), 44)
    assert 0 < m2.scan_workspace_size(L.ScanShape(b, T, D, N, 1, m2.F32, 1)) < 4 * b * D
    args = [cu(v[k]) for k in ORDER]
    y, fin = m2.scan_fwd(*args, cu(n), dt_softplus=True)
    yr, fr = R.scan(*[f64(v[k]) for k in ORDER], n)
    close(y, yr, "y")
    close(fin, fr, "final_state")
    assert m2.device_error() == 0
