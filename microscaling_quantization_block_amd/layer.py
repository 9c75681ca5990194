"""Binding of the steps around a layer's products (include/mxq_layer.h): the
root-mean-square norm with a quantized output, and its gradient.

Like decode.py: argument marshalling and host checks only, outputs and
workspaces the caller does not pass are allocated with torch, and every call is
asynchronous, on the current stream of its tensors' device or on the one given
as stream=."""

import ctypes
from typing import NamedTuple, Optional

import torch

from . import Format, Layout, lib
from .decode import _check_tensor, _launch, _p, _takes_stream

__all__ = ["RMSNorm", "mx_rmsnorm", "mx_rmsnorm_backward", "mx_rmsnorm_backward_workspace"]

_fns = None


def _lib():
    global _fns
    if _fns is None:
        L = lib()
        i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
        L.mx_rmsnorm.argtypes = [vp, i64, vp, i64, vp, i64, i64, f32, vp, i64, vp, i64, vp, i32, i32, vp, i64, vp, vp, vp,
                                 i64, vp]
        L.mx_rmsnorm_backward.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, i64, i64, vp, i64, vp, vp, i64, vp]
        L.mx_rmsnorm_backward_workspace.argtypes = [i64, i64]
        for f in ("mx_rmsnorm", "mx_rmsnorm_backward"):
            getattr(L, f).restype = ctypes.c_int
        L.mx_rmsnorm_backward_workspace.restype = i64
        _fns = L
    return _fns


def _matrix(t, name, rows, cols, dev, dtype=torch.bfloat16):
    """A [rows, cols] matrix with unit column stride; returns its row stride (that of a single row means nothing)."""
    _check_tensor(t, name, dtype, 2, dev)
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.stride(0) if rows > 1 else cols


def _flat(t, name, dtype, n, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.device != dev or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be contiguous on {dev} with {n} entries")


def _first(x, name):
    """Rows, columns and device of the matrix that a call goes by."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not x.is_cuda:
        raise TypeError(f"{name} must be a 2-D CUDA tensor")
    return x.shape[0], x.shape[1], x.device


# --------------------------------------------------------------------- the norm

class RMSNorm(NamedTuple):
    """What mx_rmsnorm gives; what was not asked for is None."""
    y: Optional[torch.Tensor]
    h: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    gscales: Optional[torch.Tensor]
    dq: Optional[torch.Tensor]


_BLOCK = {Format.MXFP8: 32, Format.NVFP4: 16, Format.FP8_B128: 128, Format.FP8_B128_F32: 128}


@_takes_stream
def mx_rmsnorm(x, weight, eps=1e-6, residual=None, fmt=Format.BF16, layout=Layout.LINEAR, with_y=False, with_dq=False,
               with_rstd=False, h=None, y=None, rstd=None, codes=None, scales=None, gscales=None, dq=None):
    """Root-mean-square norm of the BF16 rows x [rows, cols], after the
    residual's addition where one is given: h = bf16(x + residual),
    y = bf16(h rstd weight).  fmt names the output: Format.BF16 gives y; the
    others give the rowwise quantized copy of y (codes, scales and, for NVFP4,
    gscales: the bytes that mx_quantize, nvfp4_quantize, fp8bw_quantize or
    fp8bw_quantize_f32 give for y), and y too with with_y (or y=).  with_dq
    adds the codes' values in BF16, with_rstd what mx_rmsnorm_backward takes.
    Returns an RMSNorm.  h may be x or residual itself."""
    rows, cols, dev = _first(x, "x")
    fmt = Format(fmt)
    ld_x = _matrix(x, "x", rows, cols, dev)
    _flat(weight, "weight", torch.bfloat16, cols, dev)
    bf16 = lambda: torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    ld_r = ld_h = ld_y = ld_c = ld_dq = 0
    if residual is not None:
        ld_r = _matrix(residual, "residual", rows, cols, dev)
        h = bf16() if h is None else h
        ld_h = _matrix(h, "h", rows, cols, dev)
    elif h is not None:
        raise ValueError("h without a residual is x")
    if y is None and (with_y or fmt == Format.BF16):
        y = bf16()
    if y is not None:
        ld_y = _matrix(y, "y", rows, cols, dev)
    if rstd is None and with_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    elif rstd is not None:
        _flat(rstd, "rstd", torch.float32, rows, dev)
    if fmt == Format.BF16:
        if with_dq or any(t is not None for t in (codes, scales, gscales, dq)):
            raise ValueError("BF16 output has no codes")
    else:
        width = cols // 2 if fmt == Format.NVFP4 else cols
        sdt = torch.float32 if fmt == Format.FP8_B128_F32 else torch.uint8
        blocks = cols // _BLOCK[fmt]
        codes = torch.empty((rows, width), dtype=torch.uint8, device=dev) if codes is None else codes
        ld_c = _matrix(codes, "codes", rows, width, dev, torch.uint8)
        scales = torch.empty((rows, blocks), dtype=sdt, device=dev) if scales is None else scales
        _flat(scales, "scales", sdt, rows * blocks, dev)
        if fmt == Format.NVFP4:
            gscales = torch.empty(rows, dtype=torch.float32, device=dev) if gscales is None else gscales
            _flat(gscales, "gscales", torch.float32, rows, dev)
        elif gscales is not None:
            raise ValueError("gscales are NVFP4's")
        if dq is None and with_dq:
            dq = bf16()
        if dq is not None:
            ld_dq = _matrix(dq, "dq", rows, cols, dev)
    _launch(dev, _lib().mx_rmsnorm, x.data_ptr(), ld_x, _p(residual), ld_r, weight.data_ptr(), rows, cols, eps, _p(h), ld_h,
            _p(y), ld_y, _p(rstd), int(fmt), int(layout), _p(codes), ld_c, _p(scales), _p(gscales), _p(dq), ld_dq)
    return RMSNorm(y, h, rstd, codes, scales, gscales, dq)


def mx_rmsnorm_backward_workspace(rows, cols):
    """Bytes of workspace that mx_rmsnorm_backward needs for dweight."""
    return _lib().mx_rmsnorm_backward_workspace(rows, cols)


@_takes_stream
def mx_rmsnorm_backward(dy, h, weight, rstd, dresidual=None, dx=None, dweight=None, with_dweight=True, workspace=None):
    """Gradient of mx_rmsnorm: dy [rows, cols] of y, h (x without a residual)
    and rstd as the forward call left them, dresidual the gradient that reaches h
    by the residual stream.  Returns (dx, dweight): BF16 [rows, cols], the
    gradient of x and of the residual alike, and float32 [cols] (None with
    with_dweight=False).  dx may be dy or dresidual itself."""
    rows, cols, dev = _first(dy, "dy")
    ld_dy, ld_h = _matrix(dy, "dy", rows, cols, dev), _matrix(h, "h", rows, cols, dev)
    _flat(weight, "weight", torch.bfloat16, cols, dev)
    _flat(rstd, "rstd", torch.float32, rows, dev)
    ld_dr = 0 if dresidual is None else _matrix(dresidual, "dresidual", rows, cols, dev)
    dx = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev) if dx is None else dx
    ld_dx = _matrix(dx, "dx", rows, cols, dev)
    have = 0
    if dweight is None and with_dweight:
        dweight = torch.empty(cols, dtype=torch.float32, device=dev)
    if dweight is not None:
        _flat(dweight, "dweight", torch.float32, cols, dev)
        if workspace is None:
            have = _lib().mx_rmsnorm_backward_workspace(rows, cols)
            workspace = torch.empty(have, dtype=torch.uint8, device=dev)
        else:
            _check_tensor(workspace, "workspace", torch.uint8, 1, dev)
            have = workspace.numel() if workspace.is_contiguous() else 0
    _launch(dev, _lib().mx_rmsnorm_backward, dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, weight.data_ptr(), rstd.data_ptr(),
            _p(dresidual), ld_dr, rows, cols, dx.data_ptr(), ld_dx, _p(dweight), _p(workspace), have)
    return dx, dweight
