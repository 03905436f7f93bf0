"""The operators that stand around the chunked scan in a layer: a short causal
convolution (conv_fwd, conv_bwd, conv_step), a selective scan with a decay per
channel and state (scan_fwd, scan_bwd, scan_step) and a gated group norm
(norm_fwd, norm_bwd).

Binding of the C ABI in include/mamba2_layer.h, which states the formulas; argument
names and layouts are the same.  Token tensors are [b, T, D] (bf16 or fp32, each
token's values contiguous, any other strides: column slices of one projection output
need no copy); parameters and scan states are fp32.  `lengths` is an int32 [b] tensor
of real tokens per sequence: what lies behind them is never read into a result, and
outputs and gradients there are 0.  Tensors live on the current CUDA device;
everything runs on `stream` (default: the current stream), on which the tensors have
to be ready.  Outputs and workspaces are allocated with torch unless given; what is given
to be written (`state` of the step calls too) must not share memory with any other tensor
of the call, which is checked.

The checks and the call itself are native code (binding/layer_ext.cpp); there is no
CPU path.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

CONV_SILU = 1
SCAN_SOFTPLUS = 1
NORM_GATE_AFTER = 1

# Symbols of include/mamba2_layer.h (checked by the CPU test suite).
SYMBOLS = ("mamba2_conv_fwd", "mamba2_conv_step", "mamba2_conv_bwd", "mamba2_conv_bwd_workspace_size",
           "mamba2_scan_fwd", "mamba2_scan_step", "mamba2_scan_bwd", "mamba2_scan_workspace_size",
           "mamba2_scan_bwd_workspace_size", "mamba2_scan_selftest_turn_timeout", "mamba2_norm_fwd",
           "mamba2_norm_bwd", "mamba2_norm_bwd_workspace_size")

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


_strides2 = _i64 * 4   # mirror of struct mamba2_conv_strides
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
    f = lib.mamba2_scan_selftest_turn_timeout
    f.argtypes = [vp] * 9 + [sz, ctypes.c_uint32, vp]
    f.restype = ctypes.c_int
    _fns["scan_selftest"] = f
    return _fns


def _fn(name):
    return _fns[name] if _fns else _bind()[name]


_ext_module = None


def _load_ext():
    """The native binding (raises if it has not been built)."""
    global _ext_module
    from . import Mamba2Error, load
    from .build import ext_path
    load()
    path = ext_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m mamba_ssd_chunked_02_gb300.build`"
                           " (there is no CPU fallback)")
    spec = importlib.util.spec_from_file_location("layer_ext", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.set_error(Mamba2Error)
    _ext_module = mod
    return mod


def conv_fwd(x, w, bias=None, initial_state=None, lengths=None, *, silu=True, y=None, final_state=None,
             stream=None):
    """Causal depthwise convolution over tokens (mamba2_conv_fwd): returns (y, final_state).

    x [b,T,D], w [D,W] f32 (W = 2, 3, 4; w[:, W-1] meets the current token), bias [D] f32 or
    None, initial_state [b,W-1,D] (x's type, the tokens before the first, oldest first) or None."""
    return (_ext_module or _load_ext()).conv_fwd(x, w, bias, initial_state, lengths, silu, y, final_state, stream)


def conv_step(state, x, w, bias=None, *, silu=True, y=None, stream=None):
    """One token of conv_fwd (mamba2_conv_step): x [b,D] -> y [b,D]; `state` [b,W-1,D] (a
    final_state of conv_fwd) is moved on by the token in place."""
    return (_ext_module or _load_ext()).conv_step(state, x, w, bias, silu, y, stream)


def conv_bwd(x, w, bias=None, initial_state=None, dy=None, dfinal=None, lengths=None, *, silu=True, grads=None,
             workspace=None, stream=None):
    """Gradients of conv_fwd (mamba2_conv_bwd) for dL/dy = dy and dL/dfinal_state = dfinal (None
    = 0).  Returns a dict: dx [b,T,D] (x's type), dw [D,W] f32, dbias [D] f32 (None without
    bias), dinit [b,W-1,D] (None without initial_state).  `grads`: preallocated outputs."""
    return (_ext_module or _load_ext()).conv_bwd(x, w, bias, initial_state, dy, dfinal, lengths, silu, grads,
                                                 workspace, stream)


def conv_bwd_workspace_size(shape: ConvShape) -> int:
    """Bytes of workspace conv_bwd needs for a shape."""
    return _fn("conv_bwd_ws")(ctypes.addressof(shape))


def norm_bwd_workspace_size(shape: NormShape) -> int:
    """Bytes of workspace norm_bwd needs for a shape."""
    return _fn("norm_bwd_ws")(ctypes.addressof(shape))


def scan_workspace_size(shape: ScanShape) -> int:
    """Bytes of workspace scan_fwd needs for a shape (often 0)."""
    return _fn("scan_ws")(ctypes.addressof(shape))


def scan_bwd_workspace_size(shape: ScanShape) -> int:
    """Bytes of workspace scan_bwd needs for a shape."""
    return _fn("scan_bwd_ws")(ctypes.addressof(shape))


def scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_state=None, lengths=None, *,
             dt_softplus=False, y=None, final_state=None, workspace=None, stream=None):
    """Selective scan with a decay per channel and state (mamba2_scan_fwd): returns (y, final_state).

    x, dt [b,T,D], A [D,N] f32, B, C [b,T,G,N] (channel c reads group c / (D/G)), D [D] f32 or
    None, z [b,T,D] or None (y is multiplied by silu(z)), dt_bias [D] f32 or None, initial_state
    [b,D,N] f32 or None; N in {8, 16, 32, 64, 128}."""
    return (_ext_module or _load_ext()).scan_fwd(x, dt, A, B, C, D, z, dt_bias, initial_state, lengths, dt_softplus,
                                                 y, final_state, workspace, stream)


def scan_selftest_turn_timeout(x, dt, A, B, C, y, final_state, workspace, *, limit_us=2000, stream=None):
    """The failure path of scan_fwd's wait (mamba2_scan_selftest_turn_timeout): tensors as scan_fwd
    takes them, contiguous, of a shape whose rows take turns.  Sets DEVERR_CHAIN_SCAN."""
    from torch import float32 as f32

    from . import _check, _dtype_code, _ptr, _stream
    (b, T, D), (G, N), io = x.shape, B.shape[2:], x.dtype
    sh = ScanShape(b, T, D, N, G, _dtype_code(io), 0)
    space = _ptr(workspace, "workspace", workspace.dtype, workspace.shape)
    _check("mamba2_scan_selftest_turn_timeout", _fn("scan_selftest")(
        ctypes.addressof(sh), _ptr(x, "x", io, (b, T, D)), _ptr(dt, "dt", io, (b, T, D)), _ptr(A, "A", f32, (D, N)),
        _ptr(B, "B", io, (b, T, G, N)), _ptr(C, "C", io, (b, T, G, N)), _ptr(y, "y", io, (b, T, D)),
        _ptr(final_state, "final_state", f32, (b, D, N)), space, workspace.nbytes, int(limit_us), _stream(stream)))


def scan_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, *, dt_softplus=False, y=None, stream=None):
    """One token of scan_fwd (mamba2_scan_step): x, dt, z [b,D], B, C [b,G,N] -> y [b,D]; `state`
    [b,D,N] f32 (a final_state of scan_fwd) is updated in place."""
    return (_ext_module or _load_ext()).scan_step(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, y, stream)


def scan_bwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_state=None, dy=None, dfinal=None, lengths=None,
             *, dt_softplus=False, grads=None, workspace=None, stream=None):
    """Gradients of scan_fwd (mamba2_scan_bwd) for dL/dy = dy and dL/dfinal_state = dfinal (None =
    0).  Returns a dict: dx, ddt, dz [b,T,D] and dB, dC [b,T,G,N] in x's type, dA [D,N], dD [D],
    ddt_bias [D], dinit [b,D,N] f32; the entries of absent inputs are None.  `grads`:
    preallocated outputs."""
    return (_ext_module or _load_ext()).scan_bwd(x, dt, A, B, C, D, z, dt_bias, initial_state, dy, dfinal, lengths,
                                                 dt_softplus, grads, workspace, stream)


def norm_fwd(x, w=None, z=None, *, ngroups=1, eps=1e-5, gate_first=True, y=None, stream=None):
    """RMS norm over groups of channels with a SiLU gate (mamba2_norm_fwd): returns y [b,T,D].

    x [b,T,D], w [D] f32 or None (ones), z [b,T,D] or None (no gate).  gate_first: the norm of
    x silu(z), times w; else the norm of x, times w silu(z)."""
    return (_ext_module or _load_ext()).norm_fwd(x, w, z, ngroups, eps, gate_first, y, stream)


def norm_bwd(x, w=None, z=None, dy=None, *, ngroups=1, eps=1e-5, gate_first=True, grads=None, workspace=None,
             stream=None):
    """Gradients of norm_fwd (mamba2_norm_bwd) for dL/dy = dy.  Returns a dict: dx, dz [b,T,D] in
    x's type (dz None without z), dw [D] f32 (None without w).  `grads`: preallocated outputs."""
    return (_ext_module or _load_ext()).norm_bwd(x, w, z, dy, ngroups, eps, gate_first, grads, workspace, stream)
