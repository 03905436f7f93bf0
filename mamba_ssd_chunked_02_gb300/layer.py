"""The operators that stand around the chunked scan in a layer: a short causal
convolution (conv_fwd, conv_bwd, conv_step), a selective scan with a decay per
channel and state (scan_fwd, scan_bwd, scan_step) and a gated group norm
(norm_fwd, norm_bwd).

Thin ctypes binding of the C ABI in include/mamba2_layer.h, which states the
formulas; argument names and layouts are the same.  Token tensors are [b, T, D]
(bf16 or fp32, each token's values contiguous, any other strides: column slices of
one projection output need no copy); parameters and scan states are fp32.
`lengths` is an int32 [b] tensor of real tokens per sequence: what lies behind them
is never read into a result, and outputs and gradients there are 0.  Tensors live
on the current CUDA device; everything runs on `stream` (default: the current
stream), on which the tensors have to be ready.  Outputs and workspaces are
allocated with torch unless given.
"""
from __future__ import annotations

import ctypes

import torch

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
CONV_SILU = 1
SCAN_SOFTPLUS = 1
NORM_GATE_AFTER = 1

# Symbols of include/mamba2_layer.h (checked by the CPU test suite).
SYMBOLS = ("mamba2_conv_fwd", "mamba2_conv_step", "mamba2_conv_bwd", "mamba2_conv_bwd_workspace_size",
           "mamba2_scan_fwd", "mamba2_scan_step", "mamba2_scan_bwd", "mamba2_scan_workspace_size",
           "mamba2_scan_bwd_workspace_size", "mamba2_norm_fwd", "mamba2_norm_bwd",
           "mamba2_norm_bwd_workspace_size")

_i64, _i32 = ctypes.c_int64, ctypes.c_int32


class ConvShape(ctypes.Structure):
    """mirror of struct mamba2_conv_shape"""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("width", _i32), ("dtype", _i32),
                ("flags", _i32)]


class ScanShape(ctypes.Structure):
    """mirror of struct mamba2_scan_shape"""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("states", _i64), ("groups", _i64),
                ("dtype", _i32), ("flags", _i32)]


class NormShape(ctypes.Structure):
    """mirror of struct mamba2_norm_shape"""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("groups", _i64),
                ("eps", ctypes.c_float), ("dtype", _i32), ("flags", _i32)]


_strides2, _strides3, _strides6 = _i64 * 4, _i64 * 6, _i64 * 12   # {batch, token} of 2, 3, 6 tensors
_fns = {}


def _bind():
    """Argument types of the entry points, once."""
    from . import load
    lib = load()
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    for name, n in (("conv_fwd", 10), ("conv_step", 8), ("conv_bwd", 13), ("scan_fwd", 14), ("scan_step", 13),
                    ("scan_bwd", 23), ("norm_fwd", 7), ("norm_bwd", 9)):
        f = getattr(lib, "mamba2_" + name)
        spaced = name in ("conv_bwd", "scan_fwd", "scan_bwd", "norm_bwd")
        f.argtypes = [vp] * n + ([vp, sz, vp] if spaced else [])
        f.restype = ctypes.c_int
        _fns[name] = f
    for name in ("conv_bwd", "scan", "scan_bwd", "norm_bwd"):
        f = getattr(lib, "mamba2_" + name + "_workspace_size")
        f.argtypes = [vp]
        f.restype = sz
        _fns[name + "_ws"] = f
    return _fns


def _fn(name):
    return _fns[name] if _fns else _bind()[name]


def _call(name, *args):
    rc = _fn(name)(*args)
    if rc:
        from . import Mamba2Error
        raise Mamba2Error("mamba2_" + name, rc)


# The current stream's handle without a Stream object, and the current device without the
# lazy-initialisation check: 0.1 us instead of 3 us of a 10 us call.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _raw_stream(stream, device):
    """The cudaStream_t to launch on: `stream`, or the current one of `device`."""
    if stream is None:
        return _current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _io(x, name):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = x.dtype
    if d is not _BF16 and d is not _F32:
        raise TypeError(f"unsupported element type {d}: {name} must be bfloat16 or float32")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if x.get_device() != _current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return d


def _dense(t, name, dtype, shape, device, optional=False):
    """Address of a contiguous tensor."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on the same device as the input")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _token(t, name, dtype, shape, device, st, at, lead=2, optional=False):
    """Address of a token tensor; its {batch, token} strides go to st[at], st[at + 1].
    `lead` dimensions come before a token's values: 2 (batch, token) or 1 (batch)."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on the same device as the input")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    s = t.stride()
    width = shape[-1]
    if s[-1] != 1 and width > 1:
        raise ValueError(f"{name}: each token's data must be contiguous")
    if len(shape) > lead + 1:       # groups by states
        if s[-2] != width and shape[-2] > 1:
            raise ValueError(f"{name}: each token's data must be contiguous")
        width *= shape[-2]
    # a dimension of one entry is never stepped over: any stride does
    st[at] = s[0] if shape[0] > 1 else width
    st[at + 1] = s[1] if lead == 2 and shape[1] > 1 else width
    return t.data_ptr()


def _space(kind, shape, workspace, device):
    """(workspace tensor or None, its address, its bytes)."""
    need = _fn(kind + "_ws")(ctypes.addressof(shape))
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != device or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the same device as the input")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


_addr = ctypes.addressof


# ---- conv -------------------------------------------------------------------

def _conv_shape(b, T, D, w, io, silu):
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] != D:
        raise ValueError(f"w must be a [channels, width] tensor with {D} channels")
    return ConvShape(b, T, D, w.shape[1], 1 if io is _BF16 else 0, CONV_SILU if silu else 0)


def conv_fwd(x, w, bias=None, initial_state=None, lengths=None, *, silu=True, y=None, final_state=None,
             stream=None):
    """Causal depthwise convolution over tokens (mamba2_conv_fwd): returns (y, final_state).

    x [b,T,D], w [D,W] f32 (W = 2, 3, 4; w[:, W-1] meets the current token), bias [D] f32 or
    None, initial_state [b,W-1,D] (x's type, the tokens before the first, oldest first) or None."""
    io = _io(x, "x")
    b, T, D = x.shape
    dev = x.get_device()
    sh = _conv_shape(b, T, D, w, io, silu)
    W = sh.width
    if y is None:
        y = torch.empty((b, T, D), dtype=io, device=x.device)
    if final_state is None:
        final_state = torch.empty((b, W - 1, D), dtype=io, device=x.device)
    st = _strides2()
    _call("conv_fwd", _addr(sh), _addr(st), _token(x, "x", io, (b, T, D), dev, st, 0),
          _dense(w, "w", _F32, (D, W), dev), _dense(bias, "bias", _F32, (D,), dev, True),
          _dense(initial_state, "initial_state", io, (b, W - 1, D), dev, True),
          _dense(lengths, "lengths", _I32, (b,), dev, True), _token(y, "y", io, (b, T, D), dev, st, 2),
          _dense(final_state, "final_state", io, (b, W - 1, D), dev), _raw_stream(stream, dev))
    return y, final_state


def conv_step(state, x, w, bias=None, *, silu=True, y=None, stream=None):
    """One token of conv_fwd (mamba2_conv_step): x [b,D] -> y [b,D]; `state` [b,W-1,D] (a
    final_state of conv_fwd) is moved on by the token in place."""
    io = _io(x, "x")
    b, D = x.shape
    dev = x.get_device()
    sh = _conv_shape(b, 1, D, w, io, silu)
    W = sh.width
    if y is None:
        y = torch.empty((b, D), dtype=io, device=x.device)
    st = _strides2()
    _call("conv_step", _addr(sh), _addr(st), _dense(state, "state", io, (b, W - 1, D), dev),
          _token(x, "x", io, (b, D), dev, st, 0, 1), _dense(w, "w", _F32, (D, W), dev),
          _dense(bias, "bias", _F32, (D,), dev, True), _token(y, "y", io, (b, D), dev, st, 2, 1),
          _raw_stream(stream, dev))
    return y


def _grads(grads, shapes, device):
    """The outputs of a backward: given ones, and new ones for the other (shape, dtype) entries."""
    g = dict(grads or {})
    for k, v in shapes.items():
        if v is None:
            g[k] = None
        elif g.get(k) is None:
            g[k] = torch.empty(v[0], dtype=v[1], device=device)
    return g


def conv_bwd(x, w, bias=None, initial_state=None, dy=None, dfinal=None, lengths=None, *, silu=True, grads=None,
             workspace=None, stream=None):
    """Gradients of conv_fwd (mamba2_conv_bwd) for dL/dy = dy and dL/dfinal_state = dfinal (None
    = 0).  Returns a dict: dx [b,T,D] (x's type), dw [D,W] f32, dbias [D] f32 (None without
    bias), dinit [b,W-1,D] (None without initial_state).  `grads`: preallocated outputs."""
    io = _io(x, "x")
    b, T, D = x.shape
    dev = x.get_device()
    sh = _conv_shape(b, T, D, w, io, silu)
    W = sh.width
    win = (b, W - 1, D)
    g = _grads(grads, dict(dx=((b, T, D), io), dw=((D, W), _F32), dbias=((D,), _F32) if bias is not None else None,
                           dinit=(win, io) if initial_state is not None else None), x.device)
    st = _strides2()
    ws, wp, wb = _space("conv_bwd", sh, workspace, dev)
    _call("conv_bwd", _addr(sh), _addr(st), _token(x, "x", io, (b, T, D), dev, st, 0),
          _dense(w, "w", _F32, (D, W), dev), _dense(bias, "bias", _F32, (D,), dev, True),
          _dense(initial_state, "initial_state", io, win, dev, True),
          _token(dy, "dy", io, (b, T, D), dev, st, 2), _dense(dfinal, "dfinal", io, win, dev, True),
          _dense(lengths, "lengths", _I32, (b,), dev, True), _dense(g["dx"], "dx", io, (b, T, D), dev),
          _dense(g["dw"], "dw", _F32, (D, W), dev), _dense(g["dbias"], "dbias", _F32, (D,), dev, True),
          _dense(g["dinit"], "dinit", io, win, dev, True), wp, wb, _raw_stream(stream, dev))
    return g


# ---- scan -------------------------------------------------------------------

def _scan_shape(b, T, D, A, B, io, softplus):
    if not isinstance(A, torch.Tensor) or A.dim() != 2 or A.shape[0] != D:
        raise ValueError(f"A must be a [channels, states] tensor with {D} channels")
    if not isinstance(B, torch.Tensor) or B.dim() < 3:
        raise ValueError("B must be a [.., groups, states] tensor")
    return ScanShape(b, T, D, A.shape[1], B.shape[-2], 1 if io is _BF16 else 0, SCAN_SOFTPLUS if softplus else 0)


def scan_workspace_size(shape: ScanShape) -> int:
    """Bytes of workspace scan_fwd needs for a shape (often 0)."""
    return _fn("scan_ws")(_addr(shape))


def scan_bwd_workspace_size(shape: ScanShape) -> int:
    """Bytes of workspace scan_bwd needs for a shape."""
    return _fn("scan_bwd_ws")(_addr(shape))


def scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_state=None, lengths=None, *,
             dt_softplus=False, y=None, final_state=None, workspace=None, stream=None):
    """Selective scan with a decay per channel and state (mamba2_scan_fwd): returns (y, final_state).

    x, dt [b,T,D], A [D,N] f32, B, C [b,T,G,N] (channel c reads group c / (D/G)), D [D] f32 or
    None, z [b,T,D] or None (y is multiplied by silu(z)), dt_bias [D] f32 or None, initial_state
    [b,D,N] f32 or None; N in {8, 16, 32, 64, 128}."""
    io = _io(x, "x")
    b, T, ch = x.shape
    dev = x.get_device()
    sh = _scan_shape(b, T, ch, A, B, io, dt_softplus)
    N, G = sh.states, sh.groups
    if y is None:
        y = torch.empty((b, T, ch), dtype=io, device=x.device)
    if final_state is None:
        final_state = torch.empty((b, ch, N), dtype=_F32, device=x.device)
    tok, bc = (b, T, ch), (b, T, G, N)
    st = _strides6()
    ws, wp, wb = _space("scan", sh, workspace, dev)
    _call("scan_fwd", _addr(sh), _addr(st), _token(x, "x", io, tok, dev, st, 0), _token(dt, "dt", io, tok, dev, st, 2),
          _dense(A, "A", _F32, (ch, N), dev), _token(B, "B", io, bc, dev, st, 4), _token(C, "C", io, bc, dev, st, 6),
          _dense(D, "D", _F32, (ch,), dev, True), _token(z, "z", io, tok, dev, st, 8, 2, True),
          _dense(dt_bias, "dt_bias", _F32, (ch,), dev, True),
          _dense(initial_state, "initial_state", _F32, (b, ch, N), dev, True),
          _dense(lengths, "lengths", _I32, (b,), dev, True), _token(y, "y", io, tok, dev, st, 10),
          _dense(final_state, "final_state", _F32, (b, ch, N), dev), wp, wb, _raw_stream(stream, dev))
    return y, final_state


def scan_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, *, dt_softplus=False, y=None, stream=None):
    """One token of scan_fwd (mamba2_scan_step): x, dt, z [b,D], B, C [b,G,N] -> y [b,D]; `state`
    [b,D,N] f32 (a final_state of scan_fwd) is updated in place."""
    io = _io(x, "x")
    b, ch = x.shape
    dev = x.get_device()
    sh = _scan_shape(b, 1, ch, A, B, io, dt_softplus)
    N, G = sh.states, sh.groups
    if y is None:
        y = torch.empty((b, ch), dtype=io, device=x.device)
    tok, bc = (b, ch), (b, G, N)
    st = _strides6()
    _call("scan_step", _addr(sh), _addr(st), _dense(state, "state", _F32, (b, ch, N), dev),
          _token(x, "x", io, tok, dev, st, 0, 1), _token(dt, "dt", io, tok, dev, st, 2, 1),
          _dense(A, "A", _F32, (ch, N), dev), _token(B, "B", io, bc, dev, st, 4, 1),
          _token(C, "C", io, bc, dev, st, 6, 1), _dense(D, "D", _F32, (ch,), dev, True),
          _token(z, "z", io, tok, dev, st, 8, 1, True), _dense(dt_bias, "dt_bias", _F32, (ch,), dev, True),
          _token(y, "y", io, tok, dev, st, 10, 1), _raw_stream(stream, dev))
    return y


def scan_bwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_state=None, dy=None, dfinal=None, lengths=None,
             *, dt_softplus=False, grads=None, workspace=None, stream=None):
    """Gradients of scan_fwd (mamba2_scan_bwd) for dL/dy = dy and dL/dfinal_state = dfinal (None =
    0).  Returns a dict: dx, ddt, dz [b,T,D] and dB, dC [b,T,G,N] in x's type, dA [D,N], dD [D],
    ddt_bias [D], dinit [b,D,N] f32; the entries of absent inputs are None.  `grads`:
    preallocated outputs."""
    io = _io(x, "x")
    b, T, ch = x.shape
    dev = x.get_device()
    sh = _scan_shape(b, T, ch, A, B, io, dt_softplus)
    N, G = sh.states, sh.groups
    tok, bc, hs = (b, T, ch), (b, T, G, N), (b, ch, N)
    g = _grads(grads, dict(dx=(tok, io), ddt=(tok, io), dA=((ch, N), _F32), dB=(bc, io), dC=(bc, io),
                           dD=((ch,), _F32) if D is not None else None, dz=(tok, io) if z is not None else None,
                           ddt_bias=((ch,), _F32) if dt_bias is not None else None,
                           dinit=(hs, _F32) if initial_state is not None else None), x.device)
    st = _strides6()
    ws, wp, wb = _space("scan_bwd", sh, workspace, dev)
    _call("scan_bwd", _addr(sh), _addr(st), _token(x, "x", io, tok, dev, st, 0), _token(dt, "dt", io, tok, dev, st, 2),
          _dense(A, "A", _F32, (ch, N), dev), _token(B, "B", io, bc, dev, st, 4), _token(C, "C", io, bc, dev, st, 6),
          _dense(D, "D", _F32, (ch,), dev, True), _token(z, "z", io, tok, dev, st, 8, 2, True),
          _dense(dt_bias, "dt_bias", _F32, (ch,), dev, True),
          _dense(initial_state, "initial_state", _F32, hs, dev, True), _token(dy, "dy", io, tok, dev, st, 10),
          _dense(dfinal, "dfinal", _F32, hs, dev, True), _dense(lengths, "lengths", _I32, (b,), dev, True),
          _dense(g["dx"], "dx", io, tok, dev), _dense(g["ddt"], "ddt", io, tok, dev),
          _dense(g["dA"], "dA", _F32, (ch, N), dev), _dense(g["dB"], "dB", io, bc, dev),
          _dense(g["dC"], "dC", io, bc, dev), _dense(g["dD"], "dD", _F32, (ch,), dev, True),
          _dense(g["dz"], "dz", io, tok, dev, True), _dense(g["ddt_bias"], "ddt_bias", _F32, (ch,), dev, True),
          _dense(g["dinit"], "dinit", _F32, hs, dev, True), wp, wb, _raw_stream(stream, dev))
    return g


# ---- norm -------------------------------------------------------------------

def _norm_shape(x, io, ngroups, eps, gate_first):
    b, T, D = x.shape
    return NormShape(b, T, D, ngroups, eps, 1 if io is _BF16 else 0, 0 if gate_first else NORM_GATE_AFTER)


def norm_fwd(x, w=None, z=None, *, ngroups=1, eps=1e-5, gate_first=True, y=None, stream=None):
    """RMS norm over groups of channels with a SiLU gate (mamba2_norm_fwd): returns y [b,T,D].

    x [b,T,D], w [D] f32 or None (ones), z [b,T,D] or None (no gate).  gate_first: the norm of
    x silu(z), times w; else the norm of x, times w silu(z)."""
    io = _io(x, "x")
    tok = tuple(x.shape)
    dev = x.get_device()
    sh = _norm_shape(x, io, ngroups, eps, gate_first)
    if y is None:
        y = torch.empty(tok, dtype=io, device=x.device)
    st = _strides3()
    _call("norm_fwd", _addr(sh), _addr(st), _token(x, "x", io, tok, dev, st, 0),
          _dense(w, "w", _F32, tok[2:], dev, True), _token(z, "z", io, tok, dev, st, 2, 2, True),
          _token(y, "y", io, tok, dev, st, 4), _raw_stream(stream, dev))
    return y


def norm_bwd(x, w=None, z=None, dy=None, *, ngroups=1, eps=1e-5, gate_first=True, grads=None, workspace=None,
             stream=None):
    """Gradients of norm_fwd (mamba2_norm_bwd) for dL/dy = dy.  Returns a dict: dx, dz [b,T,D] in
    x's type (dz None without z), dw [D] f32 (None without w).  `grads`: preallocated outputs."""
    io = _io(x, "x")
    tok = tuple(x.shape)
    dev = x.get_device()
    sh = _norm_shape(x, io, ngroups, eps, gate_first)
    g = _grads(grads, dict(dx=(tok, io), dz=(tok, io) if z is not None else None,
                           dw=(tok[2:], _F32) if w is not None else None), x.device)
    st = _strides3()
    ws, wp, wb = _space("norm_bwd", sh, workspace, dev)
    _call("norm_bwd", _addr(sh), _addr(st), _token(x, "x", io, tok, dev, st, 0),
          _dense(w, "w", _F32, tok[2:], dev, True), _token(z, "z", io, tok, dev, st, 2, 2, True),
          _token(dy, "dy", io, tok, dev, st, 4), _dense(g["dx"], "dx", io, tok, dev),
          _dense(g["dz"], "dz", io, tok, dev, True), _dense(g["dw"], "dw", _F32, tok[2:], dev, True), wp, wb,
          _raw_stream(stream, dev))
    return g
