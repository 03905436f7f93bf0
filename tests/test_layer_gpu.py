"""Layer operators on the GPU against plain fp64 implementations.

Bounds, from the arithmetic: fp32 results are chains of a few hundred fp32 operations
whose relative errors (2^-24 each; the hardware exponential and reciprocal 2^-22) add up
like a random walk: below 3e-6 of the result's scale, held to 2e-5.  The scale is the
value's own size plus the tensor's rms, as sums cancel.  bf16 results carry one rounding
more, at most 2^-8 of the value's size.  Values that only move are equal."""
import pytest
import torch

import layer_ref as R
import mamba_ssd_chunked_02_gb300 as m2

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")


def close(got, want, what):
    assert got is not None and tuple(got.shape) == tuple(want.shape), what
    g, w = got.detach().double().cpu(), want.double()
    if not w.numel():
        return
    bound = 2e-5 * (w.abs() + w.square().mean().sqrt()) + (2 ** -8 * w.abs() if got.dtype == BF16 else 0) + 1e-30
    bad = ~((g - w).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((g - w).abs() / bound).max():.3g} bounds"


class Gen:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def randn(self, *shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(dtype)


def f64(v):
    return v.double() if v is not None else None


def cu(v):
    return v.cuda() if v is not None else None


def spoil(v, lengths):
    """A copy with NaN and infinities behind each sequence's length."""
    if v is None or lengths is None:
        return v
    v = v.clone()
    for i, n in enumerate(lengths.tolist()):
        v[i, n:] = NAN
        v[i, n + 1::2] = float("inf")
    return v


def pitched(v, pad, lead=0):
    """The same values as a column slice of a wider tensor on the GPU."""
    wide = torch.full((*v.shape[:-1], v.shape[-1] + pad + lead), NAN, dtype=v.dtype, device="cuda")
    out = wide[..., lead:lead + v.shape[-1]]
    out.copy_(v)
    return out


def lens(ragged, b, T):
    return torch.tensor([(T, 0, max(T - 1, 0), T // 2, 1)[i % 5] if T else 0 for i in range(b)],
                        dtype=torch.int32) if ragged else None


# ---- conv ---------------------------------------------------------------------------------------

CONV = [  # b, T, D, W, dtype, act, bias, init, ragged, pad, lead
    (1, 1, 1, 2, F32, True, True, False, False, 0, 0),
    (2, 2, 5, 4, BF16, True, True, True, False, 0, 0),
    (5, 9, 8, 4, BF16, True, True, True, True, 0, 0),
    (5, 9, 8, 3, F32, False, True, True, True, 0, 0),
    (2, 130, 264, 4, BF16, True, False, False, False, 8, 8),
    (2, 130, 263, 4, BF16, True, True, True, False, 1, 1),
    (1, 700, 40, 3, F32, True, True, False, False, 4, 4),
    (5, 67, 36, 2, F32, True, True, True, True, 2, 1),
    (5, 3, 16, 4, F32, True, True, True, True, 0, 0),
    (3, 1100, 12, 4, BF16, True, True, True, True, 0, 0),
    (2, 0, 8, 4, BF16, True, True, True, False, 0, 0),
    (1, 0, 3, 3, F32, True, True, False, False, 0, 0),
]


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(case):
    b, T, D, W, dt, act, with_bias, with_init, ragged, pad, lead = case
    r = Gen(7)
    x, w = r.randn(b, T, D, dtype=dt), r.randn(D, W, scale=0.5)
    bias = r.randn(D, scale=0.5) if with_bias else None
    init = r.randn(b, W - 1, D, dtype=dt) if with_init else None
    dy, df = r.randn(b, T, D, dtype=dt), r.randn(b, W - 1, D, dtype=dt)
    n = lens(ragged, b, T)
    xd, dyd = pitched(spoil(x, n), pad, lead), pitched(spoil(dy, n), pad, lead)
    y, fin = m2.conv_fwd(xd, cu(w), cu(bias), cu(init), cu(n), silu=act)
    yr, fr = R.conv(f64(x), f64(w), f64(bias), f64(init), n, act)
    close(y, yr, "y")
    assert torch.equal(fin.cpu().double(), fr)
    if n is not None:
        for i, k in enumerate(n.tolist()):
            assert not y[i, k:].any()
    g = m2.conv_bwd(xd, cu(w), cu(bias), cu(init), dyd, cu(df), cu(n), silu=act)
    want = R.conv(f64(x), f64(w), f64(bias), f64(init), n, act, f64(dy), f64(df))
    for k in want:
        if (k == "dbias" and bias is None) or (k == "dinit" and init is None):
            assert g[k] is None
        else:
            close(g[k], want[k], k)
    again = m2.conv_bwd(xd, cu(w), cu(bias), cu(init), dyd, cu(df), cu(n), silu=act)
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None)


@pytest.mark.parametrize("b,D,W,dt,act", [(1, 1, 2, F32, True), (3, 37, 4, BF16, True), (4, 640, 4, BF16, True),
                                          (2, 130, 3, F32, False), (257, 8, 3, BF16, True)])
def test_conv_step_continues_the_prompt(b, D, W, dt, act):
    r = Gen(8)
    T, tail = 6, 5
    x, w, bias = r.randn(b, T + tail, D, dtype=dt), r.randn(D, W, scale=0.5), r.randn(D, scale=0.5)
    whole, fin = m2.conv_fwd(cu(x), cu(w), cu(bias), silu=act)
    _, state = m2.conv_fwd(cu(x[:, :T]), cu(w), cu(bias), silu=act)
    for t in range(T, T + tail):
        xt = pitched(x[:, t], 3 if t % 2 else 8)
        close(m2.conv_step(state, xt, cu(w), cu(bias), silu=act),
              R.conv(f64(x[:, :t + 1]), f64(w), f64(bias), None, None, act)[0][:, t], f"token {t}")
    assert torch.equal(state, fin)


def test_conv_broadcast_and_transposed_inputs():
    r = Gen(9)
    w, bias = r.randn(24, 4, scale=0.5), r.randn(24)
    x = r.randn(7, 3, 24)                                   # tokens outermost
    y, _ = m2.conv_fwd(cu(x).transpose(0, 1), cu(w), cu(bias))
    close(y, R.conv(f64(x).transpose(0, 1), f64(w), f64(bias), None, None)[0], "transposed")
    one = r.randn(1, 7, 24)
    y, _ = m2.conv_fwd(cu(one).expand(3, 7, 24), cu(w), cu(bias))
    close(y, R.conv(f64(one).expand(3, 7, 24), f64(w), f64(bias), None, None)[0], "broadcast")


# ---- scan ---------------------------------------------------------------------------------------

SCAN = [  # b, T, D, N, G, dtype, softplus, D, z, bias, init, ragged, pad
    (1, 1, 1, 8, 1, F32, True, True, True, True, False, False, 0),
    (2, 7, 6, 16, 2, BF16, True, True, True, True, True, False, 0),
    (5, 37, 10, 16, 1, F32, True, True, True, True, True, True, 0),
    (5, 37, 10, 8, 2, BF16, True, True, False, True, True, True, 2),
    (1, 300, 34, 16, 1, F32, True, True, True, True, True, False, 0),
    (2, 130, 33, 16, 1, BF16, True, True, True, True, False, False, 1),
    (2, 70, 40, 32, 2, F32, True, False, True, False, True, False, 0),
    (1, 200, 20, 64, 1, BF16, True, True, True, True, True, False, 4),
    (5, 131, 6, 128, 2, F32, True, True, True, True, True, True, 0),
    (1, 129, 9, 128, 1, BF16, True, True, False, True, False, False, 0),
    (1, 513, 132, 16, 1, F32, False, True, True, True, True, False, 0),
    (3, 70, 260, 8, 1, F32, True, True, True, True, True, True, 0),
    (2, 0, 4, 16, 1, BF16, True, True, True, True, True, False, 0),
    (1, 0, 4, 16, 1, F32, True, True, True, True, False, False, 0),
]


def scan_inputs(case, seed=11):
    b, T, D, N, G, dt, softplus, with_D, gate, with_bias, with_init, ragged, pad = case
    r = Gen(seed)
    v = dict(x=r.randn(b, T, D, dtype=dt), dt=r.randn(b, T, D, dtype=dt, scale=0.5),
             A=-torch.arange(1, N + 1).float() * torch.exp(r.randn(D, N, scale=0.2)),
             B=r.randn(b, T, G, N, dtype=dt), C=r.randn(b, T, G, N, dtype=dt),
             D=r.randn(D) if with_D else None, z=r.randn(b, T, D, dtype=dt) if gate else None,
             dt_bias=r.randn(D, scale=0.5) - 3 if with_bias else None,
             init=r.randn(b, D, N, scale=0.5) if with_init else None)
    if not softplus:
        v["dt"] = (0.05 + 0.1 * torch.rand(b, T, D, generator=r.g)).to(dt)
        v["dt_bias"] = None
    return v, lens(ragged, b, T), r


ORDER = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init")


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan(case):
    b, T, D, N, G, dt, softplus = case[:7]
    pad = case[-1]
    v, n, r = scan_inputs(case)
    dy, df = r.randn(b, T, D, dtype=dt), r.randn(b, D, N)
    dev = {k: cu(v[k]) for k in ORDER}
    for k in ("x", "dt", "z"):
        if v[k] is not None:
            dev[k] = pitched(spoil(v[k], n), pad, pad)
    for k in ("B", "C"):
        dev[k] = pitched(spoil(v[k], n).flatten(2), pad, pad).unflatten(2, (G, N))
    dyd = pitched(spoil(dy, n), pad, pad)
    args = [dev[k] for k in ORDER]
    y, fin = m2.scan_fwd(*args, cu(n), dt_softplus=softplus)
    ref = [f64(v[k]) for k in ORDER]
    yr, fr = R.scan(*ref, n, softplus)
    close(y, yr, "y")
    close(fin, fr, "final_state")
    if n is not None:
        for i, k in enumerate(n.tolist()):
            assert not y[i, k:].any()
            if k == 0:
                assert torch.equal(fin[i].cpu(), v["init"][i])
    g = m2.scan_bwd(*args, dyd, cu(df), cu(n), dt_softplus=softplus)
    want = R.scan(*ref, n, softplus, f64(dy), f64(df))
    absent = dict(dD=v["D"], dz=v["z"], ddt_bias=v["dt_bias"], dinit=v["init"])
    for k in want:
        if k in absent and absent[k] is None:
            assert g[k] is None
        else:
            close(g[k], want[k], k)
    again = m2.scan_bwd(*args, dyd, cu(df), cu(n), dt_softplus=softplus)
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None)


def test_scan_long_axis_is_split_and_joined():
    """Few rows and many tokens: the stretches run side by side."""
    case = (1, 2500, 20, 16, 1, F32, True, True, True, True, True, False, 0)
    v, n, r = scan_inputs(case, 12)
    sh = m2.layer.ScanShape(1, 2500, 20, 16, 1, m2.F32, 1)
    assert m2.scan_workspace_size(sh) > 0
    dy, df = r.randn(1, 2500, 20), r.randn(1, 20, 16)
    args = [cu(v[k]) for k in ORDER]
    y, fin = m2.scan_fwd(*args, dt_softplus=True)
    ref = [f64(v[k]) for k in ORDER]
    yr, fr = R.scan(*ref, None)
    close(y, yr, "y")
    close(fin, fr, "final_state")
    g, want = m2.scan_bwd(*args, cu(dy), cu(df), dt_softplus=True), R.scan(*ref, None, True, f64(dy), f64(df))
    for k in want:
        close(g[k], want[k], k)


@pytest.mark.parametrize("b,T,D,N,dt,ragged", [(40, 300, 1000, 16, BF16, False), (9, 515, 1100, 64, F32, True)])
def test_scan_rows_in_turns(b, T, D, N, dt, ragged):
    """More rows than the GPU holds: slices of the token axis hand the state on."""
    v, n, _ = scan_inputs((b, T, D, N, 1, dt, True, True, True, True, True, ragged, 0), 15)
    sh = m2.layer.ScanShape(b, T, D, N, 1, m2.BF16 if dt == BF16 else m2.F32, 1)
    assert 0 < m2.scan_workspace_size(sh) < 4 * b * D      # a word a row, no states
    args = [cu(v[k]) for k in ORDER]
    runs = [m2.scan_fwd(*args, cu(n), dt_softplus=True) for _ in range(3)]
    yr, fr = R.scan(*[f64(v[k]) for k in ORDER], n)
    close(runs[0][0], yr, "y")
    close(runs[0][1], fr, "final_state")
    assert all(torch.equal(y, runs[0][0]) and torch.equal(f, runs[0][1]) for y, f in runs)
    assert m2.device_error() == 0


def test_scan_strong_and_absent_decay():
    """Steps that wipe the state out (exp(dA) = 0), steps of almost 0, and no decay (A = 0)."""
    case = (1, 50, 4, 16, 1, F32, True, True, False, False, True, False, 0)
    v, _, r = scan_inputs(case, 13)
    v["dt"][0, ::3], v["dt"][0, 1::3] = 40.0, -40.0
    v["A"][:, 8:] = 0
    args, ref = [cu(v[k]) for k in ORDER], [f64(v[k]) for k in ORDER]
    y, fin = m2.scan_fwd(*args, dt_softplus=True)
    yr, fr = R.scan(*ref, None)
    close(y, yr, "y")
    close(fin, fr, "final_state")


@pytest.mark.parametrize("b,D,N,G,dt,gate", [(1, 1, 8, 1, F32, True), (3, 30, 16, 2, BF16, True),
                                             (2, 20, 32, 1, F32, False), (9, 12, 64, 4, BF16, True),
                                             (2, 5, 128, 1, F32, True)])
def test_scan_step_continues_the_prompt(b, D, N, G, dt, gate):
    T, tail = 5, 3
    case = (b, T + tail, D, N, G, dt, True, True, gate, True, True, False, 0)
    v, _, r = scan_inputs(case, 14)
    ref = [f64(v[k]) for k in ORDER]
    yr, fr = R.scan(*ref, None)
    cut = {k: (v[k][:, :T] if k in ("x", "dt", "B", "C", "z") and v[k] is not None else v[k]) for k in ORDER}
    _, state = m2.scan_fwd(*[cu(cut[k]) for k in ORDER], dt_softplus=True)
    for t in range(T, T + tail):
        tok = {k: (v[k][:, t] if v[k] is not None else None) for k in ("x", "dt", "B", "C", "z")}
        y = m2.scan_step(state, pitched(tok["x"], 3), cu(tok["dt"]), cu(v["A"]), cu(tok["B"]), cu(tok["C"]),
                         cu(v["D"]), cu(tok["z"]), cu(v["dt_bias"]), dt_softplus=True)
        close(y, yr[:, t], f"token {t}")
    close(state, fr, "state")


# ---- norm ---------------------------------------------------------------------------------------

NORM = [  # b, T, D, G, dtype, gate, weight, pad
    (1, 1, 1, 1, F32, "first", True, 0),
    (2, 3, 21, 3, BF16, "first", True, 1),
    (2, 5, 256, 1, BF16, "first", True, 8),
    (3, 4, 1280, 2, BF16, "first", True, 0),
    (3, 4, 1280, 2, F32, "after", True, 0),
    (2, 3, 2048, 1, BF16, "after", False, 0),
    (2, 2, 5120, 1, BF16, "first", True, 0),
    (1, 3, 5121, 1, F32, None, True, 3),
    (1, 2, 20000, 1, BF16, "first", True, 0),
    (1, 3, 9001, 1, BF16, "after", True, 0),
    (1, 700, 64, 2, F32, "first", True, 0),
    (0, 4, 16, 1, F32, "first", True, 0),
    (2, 0, 16, 1, BF16, None, True, 0),
]


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm(case):
    b, T, D, G, dt, gate, weight, pad = case
    r = Gen(21)
    x, dy = r.randn(b, T, D, dtype=dt), r.randn(b, T, D, dtype=dt)
    z = r.randn(b, T, D, dtype=dt) if gate else None
    w = 1 + r.randn(D, scale=0.1) if weight else None
    first = gate != "after"
    xd, zd, dyd = pitched(x, pad, pad), pitched(z, pad, pad) if gate else None, pitched(dy, pad, pad)
    y = m2.norm_fwd(xd, cu(w), zd, ngroups=G, eps=1e-5, gate_first=first)
    close(y, R.norm(f64(x), f64(w), f64(z), G, 1e-5, first), "y")
    g = m2.norm_bwd(xd, cu(w), zd, dyd, ngroups=G, eps=1e-5, gate_first=first)
    want = R.norm(f64(x), f64(w), f64(z), G, 1e-5, first, f64(dy))
    for k in ("dx", "dz", "dw"):
        if (k == "dz" and z is None) or (k == "dw" and w is None):
            assert g[k] is None
        else:
            close(g[k], want[k], k)


def test_norm_rows_of_zeros_and_large_values():
    x = torch.zeros(1, 3, 64)
    x[0, 1] = 1e18
    x[0, 2, 5] = 1e-18
    y = m2.norm_fwd(cu(x), eps=1e-5)
    assert not y[0, 0].any()
    close(y[0, 1], torch.ones(64), "large")
    assert torch.isfinite(y).all()
    r = Gen(22)
    big, dy = r.randn(1, 2, 64) * 1e15, r.randn(1, 2, 64)      # 1 / sqrt(..) cubed underflows
    g, want = m2.norm_bwd(cu(big), None, None, cu(dy)), R.norm(f64(big), None, None, 1, 1e-5, True, f64(dy))
    close(g["dx"] * 1e15, want["dx"] * 1e15, "dx of large values")


# ---- streams, outputs given, refusals -----------------------------------------------------------

def test_given_outputs_and_another_stream():
    r = Gen(31)
    x, z, w = cu(r.randn(2, 33, 48)), cu(r.randn(2, 33, 48)), cu(r.randn(48))
    want = m2.norm_fwd(x, w, z)
    side = torch.cuda.Stream()
    wide = torch.full((2, 33, 64), 7.0, device="cuda")
    torch.cuda.synchronize()
    out = m2.norm_fwd(x, w, z, y=wide[:, :, 8:56], stream=side)
    side.synchronize()
    assert torch.equal(out, want) and (wide[:, :, :8] == 7).all() and (wide[:, :, 56:] == 7).all()
    cw = cu(r.randn(48, 4))
    want, fin = m2.conv_fwd(x, cw)
    wide.fill_(7.0)
    torch.cuda.synchronize()
    y, f2 = m2.conv_fwd(x, cw, y=wide[:, :, 8:56], stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(f2, fin) and (wide[:, :, 56:] == 7).all()


def test_another_stream_allocates_for_itself():
    """A call on a given stream takes its outputs and workspace from that stream's memory: work
    queued on the current stream before and after it does not touch them."""
    case = (1, 2500, 20, 16, 1, F32, True, True, True, True, True, False, 0)
    v, _, r = scan_inputs(case, 16)
    args = [cu(v[k]) for k in ORDER]
    dy = cu(r.randn(1, 2500, 20))
    want, fin = m2.scan_fwd(*args, dt_softplus=True)
    grads = m2.scan_bwd(*args, dy, dt_softplus=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        y, f = m2.scan_fwd(*args, dt_softplus=True, stream=side)
        g = m2.scan_bwd(*args, dy, dt_softplus=True, stream=side)
        torch.full((1 << 20,), NAN, device="cuda")          # would land in a workspace given back too early
        side.synchronize()
        assert torch.equal(y, want) and torch.equal(f, fin)
        assert all(torch.equal(g[k], grads[k]) for k in g if g[k] is not None)
        del y, f, g


def test_lengths_out_of_range_are_clamped():
    r = Gen(33)
    x, w = cu(r.randn(3, 7, 8)), cu(r.randn(8, 4))
    n, m = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([-5, 100, 2 ** 31 - 1], [0, 7, 7]))
    for a, b in zip(m2.conv_fwd(x, w, lengths=n), m2.conv_fwd(x, w, lengths=m)):
        assert torch.equal(a, b)
    A, B = -torch.rand(8, 16, device="cuda"), cu(r.randn(3, 7, 1, 16))
    for a, b in zip(m2.scan_fwd(x, x, A, B, B, lengths=n, dt_softplus=True),
                    m2.scan_fwd(x, x, A, B, B, lengths=m, dt_softplus=True)):
        assert torch.equal(a, b)


def test_steps_in_a_graph():
    """The single-token forms captured once and replayed token by token."""
    r = Gen(32)
    b, D, N = 2, 32, 16
    w, A = cu(r.randn(D, 4, scale=0.5)), -torch.rand(D, N, device="cuda")
    x, dt = cu(r.randn(b, 6, D)), cu(r.randn(b, 6, D)) - 2
    B, C = cu(r.randn(b, 6, 1, N)), cu(r.randn(b, 6, 1, N))
    xc, _ = m2.conv_fwd(x, w)
    want, fin = m2.scan_fwd(xc, dt, A, B, C, dt_softplus=True)
    win, state = torch.zeros(b, 3, D, device="cuda"), torch.zeros(b, D, N, device="cuda")
    cur = [v[:, 0].clone() for v in (x, dt, B, C)]

    def step():
        u = m2.conv_step(win, cur[0], w)
        return m2.scan_step(state, u, cur[1], A, cur[2], cur[3], dt_softplus=True)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    win.zero_()
    state.zero_()
    for t in range(6):
        for dst, src in zip(cur, (x, dt, B, C)):
            dst.copy_(src[:, t])
        graph.replay()
        close(out, want[:, t].cpu(), f"token {t}")
    close(state, fin.cpu(), "state")


def test_python_refusals():
    x, w = torch.zeros(2, 4, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    with pytest.raises(ValueError, match="each token's data"):
        m2.conv_fwd(torch.zeros(2, 4, 16, device="cuda")[:, :, ::2], w)
    with pytest.raises(ValueError, match="w must have shape|width"):
        m2.conv_fwd(x, w[:7])
    with pytest.raises(TypeError, match="bias"):
        m2.conv_fwd(x, w, torch.zeros(8, device="cuda", dtype=BF16))
    with pytest.raises(ValueError, match="initial_state"):
        m2.conv_fwd(x, w, None, torch.zeros(2, 4, 8, device="cuda"))
    with pytest.raises(TypeError, match="lengths"):
        m2.conv_fwd(x, w, None, None, torch.zeros(2, device="cuda"))
    with pytest.raises(m2.Mamba2Error, match="conv_fwd"):
        m2.conv_fwd(x, torch.zeros(8, 5, device="cuda"))
    with pytest.raises(ValueError, match="CUDA tensor"):
        m2.conv_fwd(x, w.cpu())
    A, B = torch.zeros(8, 16, device="cuda"), torch.zeros(2, 4, 1, 16, device="cuda")
    with pytest.raises(TypeError, match="dt"):
        m2.scan_fwd(x, x.to(BF16), A, B, B)
    with pytest.raises(ValueError, match="C must have shape"):
        m2.scan_fwd(x, x, A, B, B[..., :8])
    with pytest.raises(m2.Mamba2Error):
        m2.scan_fwd(x, x, A[:, :12].contiguous(), B[..., :12], B[..., :12])
    with pytest.raises(ValueError, match="dy is required"):
        m2.scan_bwd(x, x, A, B, B)
    with pytest.raises(m2.Mamba2Error):
        m2.norm_fwd(x, ngroups=3)
    with pytest.raises(m2.Mamba2Error, match="workspace"):
        m2.norm_bwd(x, w[:, 0].contiguous(), None, x, workspace=torch.zeros(4, dtype=torch.uint8, device="cuda"))
