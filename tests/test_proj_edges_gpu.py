"""Projection operators where calls go wrong: results inside wider buffers, uneven rows, far
offsets, graphs that share a workspace, calls made on another stream than the current one.
Bounds as in test_proj_gpu.py."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
import proj_ref as R
from test_proj_gpu import BF16, E4M3, F32, Gen, _operands, f64, product, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", [(7, 200, 90), (40, 130, 50), (300, 200, 90), (300, 96, 333), (520, 5000, 40)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=("f32", "bf16"))
@pytest.mark.parametrize("lead,width", [(0, 352), (16, 360), (3, 361)])
def test_result_inside_a_wider_buffer(M, K, N, dt, lead, width):
    """Rows that the copies can write whole, rows that they clip, rows that they cannot write."""
    ops, x, w = _operands(M, K, N)
    room = torch.full((M + 2, width), 7.0, device="cuda", dtype=dt)
    y = room[1:M + 1, lead:lead + N]
    assert m2.proj8_fwd(*ops, y=y) is y
    product(y, x, w.t(), "y")
    keep = room.clone()
    keep[1:M + 1, lead:lead + N] = 7
    assert (keep == 7).all()
    assert m2.device_error() == 0


@pytest.mark.parametrize("M,K,N", [(130, 1152, 70), (128, 128, 640), (1, 33000, 40), (260, 33000, 24), (129, 16384, 256)])
def test_long_sums(M, K, N):
    """More contracted blocks than a block of the few rows' kernel, or an accumulator, takes."""
    ops, x, w = _operands(M, K, N)
    for dt in (F32, BF16):
        product(m2.proj8_fwd(*ops, dtype=dt), x, w.t(), "y")
    dy = Gen(1).randn(M, N)
    g = m2.proj8_bwd(dy.cuda(), *ops)
    d = f64(dy)
    product(g["dx"], R.dequant(*R.quant(d, 1, 128), 1, 128), w, "dx")
    product(g["dw"], R.dequant(*R.quant(d, 128, 1), 128, 1).t(), R.dequant(*R.quant(x, 128, 1), 128, 1), "dw")


@pytest.mark.parametrize("M,K,N", [(150, 2560, 130), (300, 4200, 260), (129, 11000, 60), (257, 5113, 77)])
def test_sums_split_between_blocks(M, K, N):
    """Few tiles with long sums: two, four or eight pairs of blocks a tile, shares of unequal length;
    operands with the contracted index inside (y), outside (dw) and one of each (dx)."""
    ops, x, w = _operands(M, K, N, 30)
    for dt in (F32, BF16):
        y = m2.proj8_fwd(*ops, dtype=dt)
        product(y, x, w.t(), "y")
        assert torch.equal(y, m2.proj8_fwd(*ops, dtype=dt))
    # the same sizes in turn: K tokens, K outputs
    ops, x, w = _operands(K, M, N, 31)
    dy = Gen(32).randn(K, N)
    got = [m2.proj8_bwd(dy.cuda(), *ops, need_dx=False)["dw"] for _ in range(2)]
    product(got[0], R.dequant(*R.quant(f64(dy), 128, 1), 128, 1).t(), R.dequant(*R.quant(x, 128, 1), 128, 1), "dw")
    assert torch.equal(got[0], got[1])
    ops, x, w = _operands(M, N, K, 33)
    for dt in (F32, BF16):
        dy = Gen(34).randn(M, K, dtype=dt)
        dx = m2.proj8_bwd(dy.cuda(), *ops, need_dw=False)["dx"]
        product(dx, R.dequant(*R.quant(f64(dy), 1, 128), 1, 128), w, "dx")
    assert m2.device_error() == 0


@pytest.mark.parametrize("K", [64, 131])
@pytest.mark.parametrize("low,high", [(-100, 7), (-127, -105), (-9, 30), (-127, 40)])
def test_scales_of_every_size_turned(low, high, K):
    """x along its columns for dw: every e4m3 number, subnormal ones too, rows of very small and large
    scales, and of zeros with the smallest.  dw is read off with one row of dy a tile of 128."""
    r = torch.Generator().manual_seed(40)
    M = 300
    bits = torch.randint(0, 256, (M, K), generator=r).to(torch.uint8)
    bits[(bits & 127) == 127] = 5
    bits[::17] = 128
    e = torch.randint(low, high + 1, (M, 1), generator=r)
    e[::17] = -127
    room = torch.zeros(M, -(-K // 16) * 16, dtype=torch.uint8, device="cuda")
    room[:, :K] = bits.cuda()
    q = room.view(E4M3)[:, :K]
    s = (e.expand(M, -(-K // 128)) + 127).to(torch.uint8).cuda().view(torch.float8_e8m0fnu)
    x = bits.view(E4M3).double() * 2.0 ** e.double()
    want = R.dequant(*R.quant(x, 128, 1), 128, 1)
    wq, ws = m2.quant8(torch.ones(3, K, device="cuda"), group="block")
    for row in (0, 1, 130, 299):
        dy = torch.zeros(M, 3)
        dy[row, 1] = 1.0
        dw = m2.proj8_bwd(dy.cuda(), q, s, wq, ws, need_dx=False)["dw"]
        assert (dw[0] == 0).all() and (dw[2] == 0).all()
        # one product of a power of two: exact where fp32 holds it
        exact = want[row].abs() >= 2.0 ** -126
        assert torch.equal(f64(dw[1])[exact], want[row][exact]), row
        assert (f64(dw[1])[~exact].abs() <= 2.0 ** -126).all()


def test_long_sums_of_gradients():
    """dw over 20000 tokens, dx over 9000 outputs: several accumulators a result."""
    M, K, N = 20000, 140, 130
    ops, x, w = _operands(M, K, N)
    dy = Gen(2).randn(M, N)
    g = m2.proj8_bwd(dy.cuda(), *ops, need_dx=False)
    product(g["dw"], R.dequant(*R.quant(f64(dy), 128, 1), 128, 1).t(), R.dequant(*R.quant(x, 128, 1), 128, 1), "dw")
    M, K, N = 150, 130, 9000
    ops, x, w = _operands(M, K, N)
    dy = Gen(3).randn(M, N)
    g = m2.proj8_bwd(dy.cuda(), *ops, need_dw=False)
    product(g["dx"], R.dequant(*R.quant(f64(dy), 1, 128), 1, 128), w, "dx")


def test_uneven_rows():
    """Sequences cut out of longer ones: rows at two distances."""
    x = Gen(4).randn(3, 9, 260)
    q, s = m2.quant8(x.cuda()[:, 2:7])
    want = R.quant(f64(x[:, 2:7]).flatten(0, 1), 1, 128)
    same(q, want[0], "q")
    same(s, want[1], "scales")
    room = torch.zeros(3, 9, 272, dtype=torch.uint8, device="cuda").view(E4M3)
    m2.quant8(x.cuda()[:, 2:7], q=room[:, 1:6, :260], scales=s)
    same(room[:, 1:6, :260], want[0], "q")
    assert (room[:, 0].float() == 0).all() and (room[:, 6:].float() == 0).all() and (room[..., 260:].float() == 0).all()
    res, dy = Gen(5).randn(3, 9, 260), Gen(6).randn(3, 9, 260)
    y, t = m2.add_norm_fwd(x.cuda()[:, 2:7], res.cuda()[:, 1:6])
    total = x[:, 2:7] + res[:, 1:6]
    same(t, f64(total), "total")
    yy = torch.zeros(3, 9, 260, device="cuda")
    m2.add_norm_fwd(x.cuda()[:, 2:7], res.cuda()[:, 1:6], y=yy[:, 3:8], total=t)
    assert torch.equal(yy[:, 3:8], y) and (yy[:, :3] == 0).all() and (yy[:, 8:] == 0).all()
    w = torch.ones(260)
    g = m2.add_norm_bwd(total.cuda(), w.cuda(), dy.cuda()[:, 2:7], res.cuda()[:, 4:])
    dx, dw = R.add_norm_bwd(f64(total), f64(w), 1e-5, f64(dy[:, 2:7]), f64(res[:, 4:]))
    assert (f64(g["dx"]) - dx).norm() <= 1e-5 * dx.norm() and (f64(g["dw"]) - dw).norm() <= 1e-5 * dw.norm()


def test_broadcast_inputs():
    """One row for all tokens (stride 0), read in place."""
    x, row = Gen(7).randn(1, 1, 256).cuda(), Gen(8).randn(2, 5, 256).cuda()
    wide = x.expand(2, 5, 256)
    y, t = m2.add_norm_fwd(wide, row)
    assert torch.equal(t, wide + row) and torch.equal(y, m2.add_norm_fwd(wide.contiguous(), row)[0])
    a, b = m2.quant8(wide), m2.quant8(wide.contiguous())
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1].view(torch.uint8), b[1].view(torch.uint8))


def test_far_offsets():
    """Results of more than 2^31 values: the rows at both ends, and a column's sum over all."""
    M, K, N = (1 << 16) + 300, 64, (1 << 15) + 96
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(M, K, device="cuda", generator=g)
    w = torch.randn(N, K, device="cuda", generator=g)
    (q, s), (wq, ws) = m2.quant8(x), m2.quant8(w, group="block")
    assert M * N > 1 << 31
    y = m2.proj8_fwd(q, s, wq, ws)
    vw = R.dequant(f64(wq), f64(ws), 128, 128)
    for at in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        product(y[at], R.dequant(f64(q[at]), f64(s[at]), 1, 128), vw.t(), f"rows {at}")
    # the gradient's operands are as long: rows of dx at both ends
    d = m2.proj8_bwd(y, q, s, wq, ws, need_dw=False)
    for at in (slice(0, 3), slice(M - 3, M)):
        product(d["dx"][at], R.dequant(*R.quant(f64(y[at]), 1, 128), 1, 128), vw, f"dx {at}")
    big, one = y[:, :64], y.shape
    del d
    q8, s8 = m2.quant8(y)
    for at in (slice(0, 2), slice(M - 2, M)):
        want = R.quant(f64(y[at]), 1, 128)
        same(q8[at], want[0], "q")
        same(s8[at], want[1], "scales")
    del q8, s8
    n, total = m2.add_norm_fwd(y)
    want = R.add_norm(f64(y[M - 2:]), None, 1e-5)
    assert ((f64(n[M - 2:]) - want).abs() <= 2e-5 + 2 ** -8 * want.abs()).all()
    assert torch.equal(total[M - 2:], y[M - 2:])
    assert m2.device_error() == 0


def test_two_widths_at_once():
    """Calls of two sizes of one form of the gradient, from two threads on streams of their own."""
    import threading
    sizes, want, got, bad = (2560, 4096), {}, {}, []
    args = {}
    for D in sizes:
        r = Gen(20 + D)
        args[D] = [r.randn(300, D).cuda(), r.randn(D).cuda(), r.randn(300, D).cuda(), r.randn(300, D).cuda()]
        want[D] = m2.add_norm_bwd(*args[D])
    torch.cuda.synchronize()

    def work(D):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    got[D] = m2.add_norm_bwd(*args[D])
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            bad.append(e)

    threads = [threading.Thread(target=work, args=(D,)) for D in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    for D in sizes:
        assert torch.equal(got[D]["dx"], want[D]["dx"]) and torch.equal(got[D]["dw"], want[D]["dw"])


def test_graphs_that_share_a_workspace():
    """Two captured backward calls over one workspace, replayed in turn on one stream."""
    a, _, _ = _operands(300, 256, 200, 10)
    b, _, _ = _operands(140, 300, 420, 11)
    da, db = Gen(12).randn(300, 200).cuda(), Gen(13).randn(140, 420).cuda()
    wa, wb = m2.proj8_bwd(da, *a), m2.proj8_bwd(db, *b)
    need = max(m2.proj8_bwd_workspace_size(m2.Proj8Shape(300, 256, 200, 0, 0)),
               m2.proj8_bwd_workspace_size(m2.Proj8Shape(140, 300, 420, 0, 0)))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    torch.cuda.synchronize()
    for d, o in ((da, a), (db, b)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m2.proj8_bwd(d, *o, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, (wa, wb)):
        assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dw"], want["dw"])


def test_first_call_inside_a_capture():
    """A form of the product that nothing has run before, captured at once."""
    q, s = m2.quant8(Gen(14).randn(20, 64).cuda())
    wq, ws = m2.quant8(Gen(15).randn(50, 64).cuda(), group="block")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = m2.proj8_fwd(q, s, wq, ws, dtype=F32)
    g.replay()
    torch.cuda.synchronize()
    product(y, R.dequant(f64(q), f64(s), 1, 128), R.dequant(f64(wq), f64(ws), 128, 128).t(), "y")


def test_back_to_back_calls_wait_for_each_other():
    """Kernels may set themselves up while the one before ends: long chains, each call on the result
    of the call before, small and large ones in turn, give what calls with a wait between give."""
    r = Gen(16)
    w = [m2.quant8(r.randn(256, 256, scale=1 / 16).cuda(), group="block") for _ in range(6)]

    def chain(x, wait):
        out = []
        for i in range(30):
            q, s = m2.quant8(x)
            x = m2.proj8_fwd(q, s, *w[i % 6], dtype=F32)
            x, _ = m2.add_norm_fwd(x)
            out.append(x)
            if wait:
                torch.cuda.synchronize()
        return out

    for M in (1, 20, 100, 700, 5000):
        x = r.randn(M, 256).cuda()
        want = chain(x, True)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(chain(x, False), want))
    assert m2.device_error() == 0
