"""The operators around a layer's projections: the norm that takes the residual in
(add_norm_fwd, add_norm_bwd), e4m3 values with power-of-two scales (quant8) and the matrix
product of such values (proj8_fwd, proj8_bwd).

Binding of the C ABI in include/mamba2_proj.h, which states the formulas; argument names and
layouts are the same.  Token tensors are [b, T, width] or [tokens, width], each token's values
contiguous.  Values in 8 bits are a pair: q (torch.float8_e4m3fn) and its scales
(torch.float8_e8m0fnu, contiguous), one for each 128 values of a row ("row": [.., ceil(D/128)])
or for each block of 128 x 128 ("block": [ceil(N/128), ceil(K/128)]); they stand for q times
scale.  Rows of q start on 16-byte boundaries: what these functions return does, as a slice of
rows padded to 16 where D is not a multiple of 16.  The tokens of the product's x, y and dy lie at
one distance throughout (sequences cut out of longer ones do not), those of x and y not within one
another; the other operators take any distances, and read tokens that share memory in place.

Tensors live on the current CUDA device; everything runs on `stream` (default: the current
stream), on which the tensors have to be ready.  Outputs and workspaces are allocated with torch
unless given; what is given to be written must not share memory with any other tensor of the
call, which is checked.  The checks and the call itself are native code (binding/proj.h); there
is no CPU path.
"""
from __future__ import annotations

import ctypes

import torch

from . import layer as _layer

ADD_NORM_QUANT = 1
QUANT8_BLOCK = 1

# Symbols of include/mamba2_proj.h (checked by the CPU test suite).
SYMBOLS = ("mamba2_add_norm_fwd", "mamba2_add_norm_bwd", "mamba2_add_norm_bwd_workspace_size", "mamba2_quant8",
           "mamba2_proj8_fwd", "mamba2_proj8_bwd", "mamba2_proj8_bwd_workspace_size", "mamba2_proj8_selftest_timeout")

_i64, _i32 = ctypes.c_int64, ctypes.c_int32


class AddNormShape(ctypes.Structure):
    """mirror of struct mamba2_add_norm_shape"""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("eps", ctypes.c_float), ("dtype", _i32),
                ("res_dtype", _i32), ("flags", _i32)]


class Proj8Shape(ctypes.Structure):
    """mirror of struct mamba2_proj8_shape"""
    _fields_ = [("tokens", _i64), ("inputs", _i64), ("outputs", _i64), ("dtype", _i32), ("flags", _i32)]


def _size_of(name, shape):
    from . import load
    f = getattr(load(), name)
    f.argtypes, f.restype = [ctypes.c_void_p], ctypes.c_size_t
    return f(ctypes.addressof(shape))


def add_norm_bwd_workspace_size(shape: AddNormShape) -> int:
    """Bytes of workspace add_norm_bwd needs for a shape (with w)."""
    return _size_of("mamba2_add_norm_bwd_workspace_size", shape)


def proj8_bwd_workspace_size(shape: Proj8Shape) -> int:
    """Bytes of workspace proj8_bwd needs for a shape (256-byte aligned)."""
    return _size_of("mamba2_proj8_bwd_workspace_size", shape)


def _ext():
    return _layer._ext_module or _layer._load_ext()


def add_norm_fwd(x, residual=None, w=None, *, eps=1e-5, quant=False, residual_f32=False, y=None, scales=None,
                 total=None, stream=None):
    """RMS norm of x + residual (mamba2_add_norm_fwd): returns (y, total), or (q, scales, total)
    with quant, q and scales being y in 8 bits in row groups.

    x [b,T,D] bf16 or f32; residual [b,T,D] of x's type or f32, or None (total = x); w [D] f32 or
    None (ones).  total = x + residual in the residual's type, or in f32 with residual_f32 (which
    the first layer's call, that has no residual yet, needs to begin one)."""
    return _ext().add_norm_fwd(x, residual, w, eps, quant, residual_f32, y, scales, total, stream)


def add_norm_bwd(total, w=None, dy=None, dtotal=None, *, eps=1e-5, grads=None, workspace=None, stream=None):
    """Gradients of add_norm_fwd (mamba2_add_norm_bwd) for dL/dy = dy (x's type) and dL/dtotal =
    dtotal (total's type, None = 0), from the total that the forward returned.  Returns a dict:
    dx [b,T,D] in dy's type, dresidual [b,T,D] in total's type (dx itself where the types are the
    same), dw [D] f32 (None without w).  `grads`: preallocated outputs."""
    return _ext().add_norm_bwd(total, w, dy, dtotal, eps, grads, workspace, stream)


def quant8(x, *, group="row", q=None, scales=None, stream=None):
    """x to e4m3 with power-of-two scales (mamba2_quant8): returns (q, scales).  group "row" for
    activations [b,T,D] or [tokens,D], "block" for a weight [N,K]; x bf16 or f32."""
    if group not in ("row", "block"):
        raise ValueError(f'group must be "row" or "block", got {group!r}')
    return _ext().quant8(x, group == "block", q, scales, stream)


def proj8_fwd(x, x_scales, w, w_scales, *, dtype=None, y=None, stream=None):
    """Matrix product in 8 bits (mamba2_proj8_fwd): y [b,T,N] = x w^T in bf16, or in `dtype`
    (torch.bfloat16 or torch.float32).

    x [b,T,K] e4m3 with x_scales in row groups, w [N,K] e4m3 with w_scales in block groups, as
    quant8 and add_norm_fwd return them.  Prompts and single tokens alike."""
    if dtype is None:
        dtype = torch.bfloat16 if y is None else y.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"unsupported element type {dtype}: dtype must be torch.bfloat16 or torch.float32")
    return _ext().proj8_fwd(x, x_scales, w, w_scales, dtype is torch.float32, y, stream)


def proj8_selftest_timeout(x, x_scales, w, w_scales, y, *, limit_us=2000, stream=None):
    """The failure path of the product's waits (mamba2_proj8_selftest_timeout): contiguous x [tokens,K],
    w [N,K] and y [tokens,N] as proj8_fwd takes them, K a multiple of 16.  Sets DEVERR_TIMEOUT_PROJ8,
    and leaves y as it is."""
    from . import _check, _dtype_code, _ptr, _stream, load
    (M, K), N = x.shape, w.shape[0]
    if K % 16:
        raise ValueError(f"K must be a multiple of 16, got {K}")
    q, s, kb = torch.float8_e4m3fn, torch.float8_e8m0fnu, -(-K // 128)
    vp = ctypes.c_void_p
    f = ctypes.CFUNCTYPE(ctypes.c_int, *[vp] * 6, ctypes.c_uint32, vp)(("mamba2_proj8_selftest_timeout", load()))
    shape = Proj8Shape(M, K, N, _dtype_code(y.dtype), 0)
    _check("mamba2_proj8_selftest_timeout", f(
        ctypes.addressof(shape), _ptr(x, "x", q, (M, K)),
        _ptr(x_scales, "x_scales", s, (M, kb)), _ptr(w, "w", q, (N, K)), _ptr(w_scales, "w_scales", s, (-(-N // 128), kb)),
        _ptr(y, "y", y.dtype, (M, N)), int(limit_us), _stream(stream)))


def proj8_bwd(dy, x, x_scales, w, w_scales, *, need_dx=True, need_dw=True, grads=None, workspace=None, stream=None):
    """Gradients of proj8_fwd (mamba2_proj8_bwd) for dL/dy = dy [b,T,N] (bf16 or f32): a dict of
    dx [b,T,K] in dy's type and dw [N,K] f32 (None where not needed).  Both products are taken in
    8 bits: dy is rounded in groups of 128 outputs for dx, dy and x in groups of 128 tokens for
    dw.  `grads`: preallocated outputs."""
    return _ext().proj8_bwd(dy, x, x_scales, w, w_scales, need_dx, need_dw, grads, workspace, stream)
