"""Binding of the steps around a layer's products (include/mxq_layer.h): the
root-mean-square norm with a quantized output, the router of a layer with
experts, the rows of its tokens ordered by expert and back, each with its
gradient; rotary positions on the way into the NVFP4 cache.

Like decode.py: argument marshalling and host checks only, outputs and
workspaces the caller does not pass are allocated with torch, and every call is
asynchronous, on the current stream of its tensors' device or on the one given
as stream=."""

import ctypes
from typing import NamedTuple, Optional

import torch

from . import Format, Layout, lib
from .decode import _Cache, _check_requests, _check_rows, _check_tensor, _launch, _p, _takes_stream

__all__ = ["RMSNorm", "mx_rmsnorm", "mx_rmsnorm_backward", "mx_rmsnorm_backward_workspace",
           "MoERows", "MoERouting", "mx_moe_route", "mx_moe_route_backward", "mx_moe_sort", "mx_moe_workspace",
           "mx_moe_dispatch", "mx_moe_combine", "mx_moe_combine_backward", "nvfp4_rope_append"]

_fns = None


def _lib():
    global _fns
    if _fns is None:
        L = lib()
        i64, i32, vp, f64 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_double
        L.mx_rmsnorm.argtypes = [vp, i64, vp, i64, vp, i64, i64, f64, vp, i64, vp, i64, vp, i32, i32, vp, i64, vp, vp, vp,
                                 i64, vp]
        L.mx_rmsnorm_backward.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, i64, i64, vp, i64, vp, vp, i64, vp]
        L.mx_rmsnorm_backward_workspace.argtypes = [i64, i64]
        L.mx_moe_route.argtypes = [vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, i64, vp]
        L.mx_moe_route_backward.argtypes = [vp, vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, i64, vp]
        L.mx_moe_sort.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, i64, vp]
        L.mx_moe_workspace.argtypes = [i64, i32, i32]
        L.mx_moe_dispatch.argtypes = [vp, i64, i64, i64, vp, i32, vp, i64, i64, vp]
        L.mx_moe_combine.argtypes = [vp, i64, i64, vp, vp, i64, i64, i32, vp, i64, vp]
        L.mx_moe_combine_backward.argtypes = [vp, i64, vp, i64, i64, vp, vp, i64, i64, i32, vp, i64, vp, vp]
        L.nvfp4_rope_append.argtypes = [vp, i64, i64, i32, vp, i64, i64, vp, i64, i64, i64, ctypes.POINTER(_Cache), vp, i64,
                                        i64, vp, vp, i64, vp, i32, i32, f64, vp, i64, i64, vp, vp, vp]
        for f in ("nvfp4_rope_append", "mx_rmsnorm", "mx_rmsnorm_backward", "mx_moe_route", "mx_moe_route_backward", "mx_moe_sort",
                  "mx_moe_dispatch", "mx_moe_combine", "mx_moe_combine_backward"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("mx_rmsnorm_backward_workspace", "mx_moe_workspace"):
            getattr(L, f).restype = i64
        _fns = L
    return _fns


# These calls are short: a check that passes costs one function call, and an output like an input is
# torch.empty_like of it (half the time of torch.empty).

def _matrix(t, name, rows, cols, dev, dtype=torch.bfloat16):
    """A [rows, cols] matrix with unit column stride; returns its row stride (that of a single row means nothing)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == (rows, cols)):
        _check_tensor(t, name, dtype, 2, dev)
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return ld if rows > 1 else cols


def _flat(t, name, dtype, n, dev):
    """A contiguous tensor of n entries."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.numel() == n and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    raise ValueError(f"{name} must be contiguous on {dev} with {n} entries")


def _workspace(need, workspace, like):
    """A workspace and its size: the caller's, or a new one where `need` bytes are."""
    if workspace is None:
        return (like.new_empty(need, dtype=torch.uint8), need) if need else (None, 0)
    _check_tensor(workspace, "workspace", torch.uint8, 1, like.device)
    return workspace, workspace.numel() if workspace.is_contiguous() else 0


def _first(x, name):
    """Rows, columns and device of the matrix that a call goes by."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not x.is_cuda:
        raise TypeError(f"{name} must be a 2-D CUDA tensor")
    return *x.shape, x.device


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
    if type(fmt) is not Format:
        fmt = Format(fmt)
    ld_x = _matrix(x, "x", rows, cols, dev)
    _flat(weight, "weight", torch.bfloat16, cols, dev)
    ld_r = ld_h = ld_y = ld_c = ld_dq = cols
    if residual is not None:
        ld_r = _matrix(residual, "residual", rows, cols, dev)
        if h is None:
            h = torch.empty_like(x)
        else:
            ld_h = _matrix(h, "h", rows, cols, dev)
    elif h is not None:
        raise ValueError("h without a residual is x")
    if y is not None:
        ld_y = _matrix(y, "y", rows, cols, dev)
    elif with_y or fmt is Format.BF16:
        y = torch.empty_like(x)
    if rstd is not None:
        _flat(rstd, "rstd", torch.float32, rows, dev)
    elif with_rstd:
        rstd = x.new_empty(rows, dtype=torch.float32)
    if fmt is Format.BF16:
        if with_dq or any(t is not None for t in (codes, scales, gscales, dq)):
            raise ValueError("BF16 output has no codes")
    else:
        width = cols // 2 if fmt is Format.NVFP4 else cols
        sdt = torch.float32 if fmt is Format.FP8_B128_F32 else torch.uint8
        blocks = cols // _BLOCK[fmt]
        codes = x.new_empty((rows, width), dtype=torch.uint8) if codes is None else codes
        ld_c = _matrix(codes, "codes", rows, width, dev, torch.uint8)
        scales = x.new_empty((rows, blocks), dtype=sdt) if scales is None else scales
        _flat(scales, "scales", sdt, rows * blocks, dev)
        if fmt is Format.NVFP4:
            gscales = x.new_empty(rows, dtype=torch.float32) if gscales is None else gscales
            _flat(gscales, "gscales", torch.float32, rows, dev)
        elif gscales is not None:
            raise ValueError("gscales are NVFP4's")
        if dq is not None:
            ld_dq = _matrix(dq, "dq", rows, cols, dev)
        elif with_dq:
            dq = torch.empty_like(x)
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
    ld_dx, have = cols, 0
    if dx is None:
        dx = torch.empty_like(dy)
    else:
        ld_dx = _matrix(dx, "dx", rows, cols, dev)
    if dweight is not None:
        _flat(dweight, "dweight", torch.float32, cols, dev)
    elif with_dweight:
        dweight = dy.new_empty(cols, dtype=torch.float32)
    if dweight is not None:
        workspace, have = _workspace(_lib().mx_rmsnorm_backward_workspace(rows, cols), workspace, dy)
    _launch(dev, _lib().mx_rmsnorm_backward, dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, weight.data_ptr(), rstd.data_ptr(),
            _p(dresidual), ld_dr, rows, cols, dx.data_ptr(), ld_dx, _p(dweight), _p(workspace), have)
    return dx, dweight


# ------------------------------------------------------------ the experts' rows

class MoERows(NamedTuple):
    """Rows ordered by (expert, token): int32 offsets [experts + 1], the token of every row [tokens * topk] and the row
    of every slot [tokens, topk] (-1: none)."""
    offsets: torch.Tensor
    row_token: torch.Tensor
    row_of: torch.Tensor


class MoERouting(NamedTuple):
    """A router's choice: int32 experts and float32 weights [tokens, topk], and the rows as in MoERows."""
    experts: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    row_token: torch.Tensor
    row_of: torch.Tensor


def _given(t, name, shape, dtype, like):
    """An output: the caller's, of that many entries, or a new one on `like`'s device."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _flat(t, name, dtype, shape if isinstance(shape, int) else shape[0] * shape[1], like.device)
    return t


def _rows_out(T, E, k, like, offsets, row_token, row_of):
    i32 = torch.int32
    return (_given(offsets, "offsets", E + 1, i32, like), _given(row_token, "row_token", T * k, i32, like),
            _given(row_of, "row_of", (T, k), i32, like))


def _logits(t, name, T, E, dev):
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16")
    return _matrix(t, name, T, E, dev, t.dtype)


def mx_moe_workspace(tokens, num_experts, topk):
    """Bytes of workspace that mx_moe_route and mx_moe_sort need for these sizes; may be 0."""
    return _lib().mx_moe_workspace(tokens, num_experts, topk)


@_takes_stream
def mx_moe_route(logits, topk, renormalize=True, experts=None, weights=None, offsets=None, row_token=None, row_of=None,
                 workspace=None):
    """The router: the topk largest of the float32 or BF16 logits [tokens,
    experts] of every token (ties to the lower expert, -inf never chosen), their
    softmax weights (over the chosen ones, or over all experts without
    renormalize), and the tokens' rows ordered by expert.  Returns a MoERouting:
    offsets and row_token go to the grouped products as group_row_offsets and
    a_row_index or x_row_index, row_of and weights to mx_moe_combine."""
    T, E, dev = _first(logits, "logits")
    ld = _logits(logits, "logits", T, E, dev)
    experts = _given(experts, "experts", (T, topk), torch.int32, logits)
    weights = _given(weights, "weights", (T, topk), torch.float32, logits)
    offsets, row_token, row_of = _rows_out(T, E, topk, logits, offsets, row_token, row_of)
    workspace, have = _workspace(_lib().mx_moe_workspace(T, E, topk), workspace, logits)
    _launch(dev, _lib().mx_moe_route, logits.data_ptr(), logits.dtype is torch.float32, ld, T, E, topk, bool(renormalize),
            experts.data_ptr(), weights.data_ptr(), offsets.data_ptr(), row_token.data_ptr(), row_of.data_ptr(),
            _p(workspace), have)
    return MoERouting(experts, weights, offsets, row_token, row_of)


@_takes_stream
def mx_moe_route_backward(dweights, logits, experts, weights, renormalize=True, dlogits=None):
    """Gradient of mx_moe_route's weights: dlogits like the logits, from float32
    dweights [tokens, topk] and what the forward call took and gave."""
    T, E, dev = _first(logits, "logits")
    ld = _logits(logits, "logits", T, E, dev)
    if not isinstance(experts, torch.Tensor) or experts.dim() != 2:
        raise TypeError("experts must be a 2-D int32 tensor")
    k = experts.shape[1]
    _flat(experts, "experts", torch.int32, T * k, dev)
    for t, name in ((weights, "weights"), (dweights, "dweights")):
        _flat(t, name, torch.float32, T * k, dev)
    if dlogits is None:
        dlogits, ld_d = torch.empty_like(logits), E
    else:
        ld_d = _matrix(dlogits, "dlogits", T, E, dev, logits.dtype)
    _launch(dev, _lib().mx_moe_route_backward, dweights.data_ptr(), logits.data_ptr(), logits.dtype is torch.float32, ld, T,
            E, k, bool(renormalize), experts.data_ptr(), weights.data_ptr(), dlogits.data_ptr(), ld_d)
    return dlogits


@_takes_stream
def mx_moe_sort(experts, num_experts, offsets=None, row_token=None, row_of=None, workspace=None):
    """The rows of given int32 expert ids [tokens, topk], ordered by (expert,
    token): a MoERows.  An id outside [0, num_experts) has no row."""
    T, k, dev = _first(experts, "experts")
    _flat(experts, "experts", torch.int32, T * k, dev)
    offsets, row_token, row_of = _rows_out(T, num_experts, k, experts, offsets, row_token, row_of)
    workspace, have = _workspace(_lib().mx_moe_workspace(T, num_experts, k), workspace, experts)
    _launch(dev, _lib().mx_moe_sort, experts.data_ptr(), T, num_experts, k, offsets.data_ptr(), row_token.data_ptr(),
            row_of.data_ptr(), _p(workspace), have)
    return MoERows(offsets, row_token, row_of)


def _row_of(row_of, T, dev):
    if not isinstance(row_of, torch.Tensor) or row_of.dim() != 2:
        raise TypeError("row_of must be a 2-D int32 tensor")
    k = row_of.shape[1]
    _flat(row_of, "row_of", torch.int32, (row_of.shape[0] if T is None else T) * k, dev)
    return row_of.shape[0], k


@_takes_stream
def mx_moe_dispatch(x, row_of, num_rows=None, out=None):
    """rows[row_of[t, j]] = x[t] for the BF16 rows x [tokens, cols]: the experts'
    rows [num_rows, cols] in memory (num_rows: tokens * topk).  Rows that no
    slot names are left as they were: in a new tensor they hold anything, NaN included, so where slots
    have no row and a later step reads every row (a second scale per tensor), pass zeros as
    out.  Its gradient is mx_moe_combine(drows, row_of)."""
    T, cols, dev = _first(x, "x")
    ld_x = _matrix(x, "x", T, cols, dev)
    _, k = _row_of(row_of, T, dev)
    if num_rows is None:
        num_rows = out.shape[0] if isinstance(out, torch.Tensor) and out.dim() else T * k
    out = x.new_empty((num_rows, cols)) if out is None else out
    ld_out = _matrix(out, "out", num_rows, cols, dev)
    _launch(dev, _lib().mx_moe_dispatch, x.data_ptr(), ld_x, T, cols, row_of.data_ptr(), k, out.data_ptr(), ld_out, num_rows)
    return out


@_takes_stream
def mx_moe_combine(rows, row_of, weights=None, out=None):
    """out[t] = sum over j of weights[t, j] rows[row_of[t, j]] (ones without
    weights): the experts' BF16 rows back to [tokens, cols], summed in float32.  A
    token without rows gives zeros."""
    M, cols, dev = _first(rows, "rows")
    ld_rows = _matrix(rows, "rows", M, cols, dev)
    T, k = _row_of(row_of, None, dev)
    if weights is not None:
        _flat(weights, "weights", torch.float32, T * k, dev)
    out = rows.new_empty((T, cols)) if out is None else out
    ld_out = _matrix(out, "out", T, cols, dev)
    _launch(dev, _lib().mx_moe_combine, rows.data_ptr(), ld_rows, M, row_of.data_ptr(), _p(weights), T, cols, k,
            out.data_ptr(), ld_out)
    return out


@_takes_stream
def mx_moe_combine_backward(dout, rows, row_of, weights, drows=None, dweights=None):
    """Gradient of mx_moe_combine: (drows like rows, dweights float32 [tokens,
    topk]) from dout [tokens, cols].  Rows of drows that no slot names are left
    as they were, and hold anything in a new tensor; their gradient is zero: pass zeros as drows
    where a later step reads every row."""
    T, cols, dev = _first(dout, "dout")
    ld_d = _matrix(dout, "dout", T, cols, dev)
    M = rows.shape[0] if isinstance(rows, torch.Tensor) and rows.dim() else 0
    ld_rows = _matrix(rows, "rows", M, cols, dev)
    _, k = _row_of(row_of, T, dev)
    _flat(weights, "weights", torch.float32, T * k, dev)
    drows = rows.new_empty((M, cols)) if drows is None else drows
    ld_dr = _matrix(drows, "drows", M, cols, dev)
    dweights = torch.empty_like(weights) if dweights is None else dweights
    _flat(dweights, "dweights", torch.float32, T * k, dev)
    _launch(dev, _lib().mx_moe_combine_backward, dout.data_ptr(), ld_d, rows.data_ptr(), ld_rows, M, row_of.data_ptr(),
            weights.data_ptr(), T, cols, k, drows.data_ptr(), ld_dr, dweights.data_ptr())
    return drows, dweights


# ------------------------------------------------- positions, on the way to the cache

@_takes_stream
def nvfp4_rope_append(q, k, v, cache, block_table, seq_lens, inv_freq, q_offsets=None, interleaved=False, factor=1.0,
                      out=None, with_dq=False, k_dq=None, v_dq=None):
    """nvfp4_cache_append with rotary positions: the first 2 * len(inv_freq)
    values of every head of the BF16 rows q [tokens, q_heads, head_dim] and k are
    turned by position * inv_freq (float32; pairs are the two halves, or
    neighbours with interleaved), cosine and sine times `factor`; then k and v
    [tokens, heads, head_dim] are quantized into the cache.  Requests as in
    nvfp4_cache_append.  Returns the turned q (out may be q itself), or
    (q, k_dq, v_dq) with with_dq (or k_dq and v_dq); rows of no request are not written."""
    T = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() else 0
    dev, n, width, ld = _check_requests(cache, block_table, seq_lens, q_offsets, T)
    h, d = cache.num_heads, cache.head_dim
    hq, qt, qh = _check_rows(q, "q", None, d, T, dev)
    _, kt, kh = _check_rows(k, "k", h, d, T, dev)
    _, vt, vh = _check_rows(v, "v", h, d, T, dev)
    _check_tensor(inv_freq, "inv_freq", torch.float32, 1, dev)
    if not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous")
    if out is None:
        out = q.new_empty((T, hq, d))
        ot, oh = hq * d, d
    else:
        _, ot, oh = _check_rows(out, "out", hq, d, T, dev)
    if with_dq or k_dq is not None or v_dq is not None:
        for name, t in (("k_dq", k_dq), ("v_dq", v_dq)):
            if t is not None:
                _check_rows(t, name, h, d, T, dev)
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
        k_dq = k.new_empty((T, h, d)) if k_dq is None else k_dq
        v_dq = v.new_empty((T, h, d)) if v_dq is None else v_dq
    _launch(dev, _lib().nvfp4_rope_append, q.data_ptr(), qt, qh, hq, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, T,
            cache._ref, block_table.data_ptr(), ld, width, seq_lens.data_ptr(), _p(q_offsets), n, inv_freq.data_ptr(),
            2 * inv_freq.numel(), bool(interleaved), factor, out.data_ptr(), ot, oh, _p(k_dq), _p(v_dq))
    return out if k_dq is None else (out, k_dq, v_dq)
