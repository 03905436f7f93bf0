"""The gradient of add_norm where every team of the kernel takes several rows: both copies of the row
ahead in turn, sums in turn, dw added up over rows; at widths of each form (one and two units a
thread, teams of a warp and of a block, wide rows that are read again), for each pair of types.
Bounds as in test_proj_gpu.py."""
import ctypes
import sys
import threading

import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2
import proj_ref as R
from mamba_ssd_chunked_02_gb300 import proj as L
from test_proj_gpu import BF16, F32, Gen, close, f64

pytestmark = pytest.mark.gpu

# D, rows (at least four for each team that an SM may hold: 32 an SM for warps, 2048 threads for
# blocks), x's and the residual's type.  Units are 4 channels of an fp32 residual, 8 of a bf16 one;
# a warp has up to 64, a block up to 2048 of them.
FORMS = [
    (120, 20000, BF16, F32), (200, 20000, BF16, F32), (256, 20000, F32, F32), (1028, 6000, F32, F32),
    (2560, 4300, BF16, F32), (2560, 4300, F32, F32), (8192, 1300, BF16, F32), (8192, 1300, F32, F32),
    (200, 20000, BF16, BF16), (400, 20000, BF16, BF16), (2560, 4300, BF16, BF16), (8192, 2500, BF16, BF16),
    (203, 20000, BF16, F32), (2561, 4300, BF16, BF16), (16392, 1300, BF16, BF16),
]


@pytest.mark.parametrize("with_dt", [True, False], ids=("dtotal", "alone"))
@pytest.mark.parametrize("D,rows,dt,rt", FORMS, ids=lambda v: str(v).replace("torch.", ""))
def test_many_rows_a_team(D, rows, dt, rt, with_dt):
    r = Gen(D)
    total, dy = r.randn(rows, D, dtype=rt), r.randn(rows, D, dtype=dt)
    dt_ = r.randn(rows, D, dtype=rt) if with_dt else None
    w = 1 + r.randn(D, scale=0.3)
    g = m2.add_norm_bwd(total.cuda(), w.cuda(), dy.cuda(), dt_.cuda() if with_dt else None)
    d, e = f64(dt_), (f64(total), f64(w), 1e-5, f64(dy))
    dx, dw = R.add_norm_bwd(*e, d)
    size = R.add_norm_bwd_size(*e, d)
    close(g["dx"], dx, "dx", size)
    close(g["dresidual"], dx, "dresidual", size)
    close(g["dw"], dw, "dw")


@pytest.mark.parametrize("D,T,dt,rt", [(200, 1501, BF16, F32), (2560, 301, BF16, F32), (2560, 301, BF16, BF16),
                                       (8192, 181, BF16, BF16)], ids=lambda v: str(v).replace("torch.", ""))
def test_many_rows_at_uneven_distances(D, T, dt, rt):
    """Sequences cut out of longer ones, each tensor's at its own place."""
    r = Gen(D + 1)
    b = 14
    total, dy, dt_ = (r.randn(b, T + 3, D, dtype=t) for t in (rt, dt, rt))
    w = 1 + r.randn(D, scale=0.3)
    cut = total[:, :T], dy[:, 1:T + 1], dt_[:, 3:]
    g = m2.add_norm_bwd(total.cuda()[:, :T], w.cuda(), dy.cuda()[:, 1:T + 1], dt_.cuda()[:, 3:])
    e = f64(cut[0]), f64(w), 1e-5, f64(cut[1])
    dx, dw = R.add_norm_bwd(*e, f64(cut[2]))
    size = R.add_norm_bwd_size(*e, f64(cut[2]))
    close(g["dx"], dx, "dx", size)
    close(g["dresidual"], dx, "dresidual", size)
    close(g["dw"], dw, "dw")


def test_two_widths_from_two_threads_at_once():
    """Two sizes of one form of the kernel, which ask for different amounts of shared memory, called
    through the C ABI from two threads without a pause: ctypes lets the other thread run during a
    call, so that calls of both sizes are under way at once.  Every call has its own output; the
    status and the results of all of them are looked at."""
    vp = ctypes.c_void_p
    f = ctypes.CFUNCTYPE(ctypes.c_int, *[vp] * 10, ctypes.c_size_t, vp)(("mamba2_add_norm_bwd", m2.load()))
    rows, rounds, calls, sizes = 24, 40, 100, (2560, 8192)
    bad, state = [], {}
    for D in sizes:
        r = Gen(60 + D)
        ins = [r.randn(rows, D).cuda(), r.randn(D).cuda(), r.randn(rows, D).cuda(), r.randn(rows, D).cuda()]
        want = m2.add_norm_bwd(*ins)
        shape = L.AddNormShape(1, rows, D, 1e-5, m2.F32, m2.F32, 0)
        space = torch.empty(m2.add_norm_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")
        dx, dw = torch.empty(calls, rows, D, device="cuda"), torch.empty(calls, D, device="cuda")
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")
        stream = torch.cuda.Stream()
        args = [[vp(ctypes.addressof(shape)), None, *(vp(t.data_ptr()) for t in ins), vp(dx[k].data_ptr()), None,
                 vp(dw[k].data_ptr()), vp(space.data_ptr()), space.nbytes, vp(stream.cuda_stream)] for k in range(calls)]
        state[D] = shape, ins, want, space, dx, dw, wrong, stream, args
    torch.cuda.synchronize()

    def work(D):
        _, _, want, _, dx, dw, wrong, stream, args = state[D]
        try:
            with torch.cuda.stream(stream):
                for _ in range(rounds):
                    dx.zero_()
                    dw.zero_()
                    status = [f(*a) for a in args]
                    assert not any(status), status
                    wrong.add_((dx != want["dx"]).sum() + (dw != want["dw"]).sum())
                    stream.synchronize()
        except BaseException as e:
            bad.append(e)

    old = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=work, args=(D,)) for D in sizes]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(old)
    torch.cuda.synchronize()
    assert not bad, bad
    assert all(state[D][6].item() == 0 for D in sizes)
