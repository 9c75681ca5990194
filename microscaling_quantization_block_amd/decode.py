"""Binding of the decode step (include/mxq_decode.h): products of a few BF16
rows with NVFP4 weights, the paged NVFP4 cache, and attention over it.

Like the rest of the package: argument marshalling and host checks only,
outputs and workspaces the caller does not pass are allocated with torch, and
every call is asynchronous, on the current stream of its tensors' device or on
the one given as stream=."""

import ctypes
import functools

import torch

from . import Block, Operand, _Operand, _check, _check_2d, lib

__all__ = ["NVFP4Cache", "nvfp4_gemv", "nvfp4_gemv_swiglu", "nvfp4_cache_append", "nvfp4_attention",
           "nvfp4_attention_workspace"]

_fns = None


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("k_gscales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("v_gscales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("code_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("gscale_stride", ctypes.c_int64), ("num_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


def _lib():
    global _fns
    if _fns is None:
        L = lib()
        i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
        op, ca = ctypes.POINTER(_Operand), ctypes.POINTER(_Cache)
        gemv = [vp, i64, i64, op, i64, i64, i64, vp, i64, i32, vp, vp, vp]
        L.nvfp4_gemv.argtypes = gemv
        L.nvfp4_gemv_swiglu.argtypes = gemv
        L.nvfp4_cache_append.argtypes = [vp, i64, i64, vp, i64, i64, i64, ca, vp, i64, i64, vp, vp, i64, vp, vp, vp]
        L.nvfp4_attention.argtypes = [vp, i64, i64, i64, i32, ca, vp, i64, i64, vp, vp, i64, f32, i64, vp, i64, i64,
                                      vp, vp, i64, vp]
        L.nvfp4_attention_workspace.argtypes = [i64, i32, i32, i32, i32, i64, i64, i32]
        for f in ("nvfp4_gemv", "nvfp4_gemv_swiglu", "nvfp4_cache_append", "nvfp4_attention"):
            getattr(L, f).restype = ctypes.c_int
        L.nvfp4_attention_workspace.restype = i64
        _fns = L
    return _fns


def _p(t):
    return None if t is None else t.data_ptr()


def _device_calls():
    """The raw handle of a device's current stream, and the current device.  A
    decode step is many short calls, and the objects that the public functions
    put around these two cost as much as a call; they serve where torch has not
    the short ones (a build without a GPU, another version)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return raw, getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_raw_stream, _current_device = _device_calls()


def _launch(device, fn, *args):
    """Calls fn(*args, stream) on the device's current stream, with `device`
    current (a launch goes to the current device, whatever its pointers are)."""
    if device.index == _current_device():
        status = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device.index))
    if status:
        _check(status)


def _takes_stream(call):
    """Adds stream=None.  With a stream the whole call runs with it current, so
    that what the call allocates (the workspace above all, which goes back to
    the allocator at once) belongs to that stream."""
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor) and t.device != stream.device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return wrapped


def _is(t, dtype, dim, device):
    """A tensor of that kind on that device (host tensors never: device is a GPU)."""
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == dim and t.device == device


def _check_tensor(t, name, dtype, dim, device):
    if _is(t, dtype, dim, device) and t.is_cuda:
        return
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != dim:
        raise TypeError(f"{name} must be a {dim}-D {dtype} tensor")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _check_index(t, name, n, device):
    if not _is(t, torch.int32, 1, device):
        _check_tensor(t, name, torch.int32, 1, device)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} entries")


def _room(name, t, need):
    """At least `need` bytes of storage from the tensor's first element on (rows may be strided)."""
    have = t.numel() * t.element_size()
    if have < need:
        have = t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()
        if have < need:
            raise ValueError(f"{name} holds {have} bytes, {need} are read")


# ------------------------------------------------------------- few-row products

def _gemv(fn, x, w, M, N, K, weight_rows, out, group_row_offsets, x_row_index):
    _check_2d(x, torch.bfloat16, "x")
    dev = x.device
    if not isinstance(w, Operand):
        raise TypeError("w must be an Operand")
    if x.shape[1] < K:
        raise ValueError(f"x has {x.shape[1]} columns, K is {K}")
    ng = 0
    if group_row_offsets is not None:
        _check_tensor(group_row_offsets, "group_row_offsets", torch.int32, 1, dev)
        ng = group_row_offsets.numel() - 1
        if ng < 1 or not group_row_offsets.is_contiguous():
            raise ValueError("group_row_offsets must be contiguous with num_groups + 1 >= 2 entries")
    if x_row_index is not None:
        _check_index(x_row_index, "x_row_index", M, dev)
    elif x.shape[0] != M:
        raise ValueError(f"x has {x.shape[0]} rows, M is {M}")
    data, scales, gs = w.data, w.scales, w.gscales
    for name, t in (("data", data), ("scales", scales), ("gscales", gs)):
        if not isinstance(t, torch.Tensor) or t.device != dev:
            raise ValueError(f"w.{name} must be a tensor on {dev}")
    if gs.dtype is not torch.float32 or not gs.is_contiguous() or not scales.is_contiguous():
        raise TypeError("w.gscales must be contiguous float32, w.scales contiguous")
    if data.element_size() != 1 or scales.element_size() != 1 or data.stride(-1) != 1:
        raise TypeError("w.data and w.scales must be bytes, rows of w.data contiguous")
    # the device reads these without a check
    g = max(ng, 1)
    need = weight_rows * g
    if M and N and K:
        _room("w.data", data, ((need - 1) * w.ld + K) // 2)
        _room("w.scales", scales, (need // 16 if w.block == Block.TILE else need) * (K // 16))
        _room("w.gscales", gs, 4 * g)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    else:
        _check_tensor(out, "out", torch.bfloat16, 2, dev)
        if out.shape[0] < M or out.shape[1] < N or out.stride(1) != 1:
            raise ValueError(f"out must hold [{M}, {N}] with unit column stride")
    # the stride of a single row means nothing
    ld_x, ld_y = x.stride(0) if x.shape[0] > 1 else K, out.stride(0) if out.shape[0] > 1 else N
    _launch(dev, fn, x.data_ptr(), ld_x, x.shape[0], ctypes.byref(w._c()), M, N, K, out.data_ptr(), ld_y, ng,
            _p(group_row_offsets), _p(x_row_index))
    return out


@_takes_stream
def nvfp4_gemv(x, w, M, N, K, out=None, group_row_offsets=None, x_row_index=None):
    """y[M, N] = x W^T for a few BF16 rows x and an NVFP4 weight Operand w
    [N, K] (as mx_gemm's b); x is used as it is, not quantized.  Grouped calls
    take int32 group_row_offsets [groups + 1] and one weight matrix per group;
    x_row_index [M] gathers rows of x."""
    return _gemv(_lib().nvfp4_gemv, x, w, M, N, K, N, out, group_row_offsets, x_row_index)


@_takes_stream
def nvfp4_gemv_swiglu(x, w, M, inter, K, out=None, group_row_offsets=None, x_row_index=None):
    """h[M, inter] = silu(x Wg^T) * (x Wu^T) for a few BF16 rows x and an NVFP4
    gate_up Operand w (gate rows, then up rows, per group); arguments as
    nvfp4_gemv."""
    return _gemv(_lib().nvfp4_gemv_swiglu, x, w, M, inter, K, 2 * inter, out, group_row_offsets, x_row_index)


# -------------------------------------------------------------------- the cache

class NVFP4Cache:
    """K and V rows in NVFP4 pages (layout: mxq_cache in include/mxq_decode.h):
        codes    uint8   [pages, heads, page_size, head_dim / 2]
        k_scales uint8   [pages, heads, page_size, head_dim / 16]
        v_scales uint8   [pages, heads, head_dim / 16, page_size]
        gscales  float32 [pages, heads, page_size]
    contiguous inside a page; pages may lie further apart (K and V alike, as in
    an interleaved allocation)."""

    def __init__(self, k_codes, k_scales, k_gscales, v_codes, v_scales, v_gscales):
        if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4:
            raise TypeError("k_codes must be a 4-D uint8 tensor")
        pages, heads, page, half = k_codes.shape
        d = 2 * half
        want = (("k_codes", k_codes, torch.uint8, (pages, heads, page, half)),
                ("k_scales", k_scales, torch.uint8, (pages, heads, page, d // 16)),
                ("k_gscales", k_gscales, torch.float32, (pages, heads, page)),
                ("v_codes", v_codes, torch.uint8, (pages, heads, page, half)),
                ("v_scales", v_scales, torch.uint8, (pages, heads, d // 16, page)),
                ("v_gscales", v_gscales, torch.float32, (pages, heads, page)))
        for name, t, dt, shape in want:
            _check_tensor(t, name, dt, len(shape), k_codes.device)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
            if pages and not t[0].is_contiguous():
                raise ValueError(f"{name} must be contiguous inside a page")
        for a, b in ((k_codes, v_codes), (k_scales, v_scales), (k_gscales, v_gscales)):
            if pages > 1 and a.stride(0) != b.stride(0):
                raise ValueError("K and V pages must have the same stride")
        self.k_codes, self.k_scales, self.k_gscales = k_codes, k_scales, k_gscales
        self.v_codes, self.v_scales, self.v_gscales = v_codes, v_scales, v_gscales
        self.num_pages, self.num_heads, self.page_size, self.head_dim = pages, heads, page, d
        self.device = k_codes.device
        stride = lambda t: t.stride(0) if pages > 1 else t[0].numel() if pages else 0
        self._c = _Cache(_p(k_codes), _p(k_scales), _p(k_gscales), _p(v_codes), _p(v_scales), _p(v_gscales), pages,
                         stride(k_codes), stride(k_scales), stride(k_gscales), heads, page, d)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, num_pages, num_heads, page_size, head_dim, device="cuda"):
        """A cache of num_pages pages; their content is not initialised."""
        u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=device)
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=device)
        n, h, p, d = num_pages, num_heads, page_size, head_dim
        return cls(u8(n, h, p, d // 2), u8(n, h, p, d // 16), f32(n, h, p), u8(n, h, p, d // 2), u8(n, h, d // 16, p),
                   f32(n, h, p))


def _check_requests(cache, block_table, seq_lens, q_offsets, rows):
    if not isinstance(cache, NVFP4Cache):
        raise TypeError("cache must be an NVFP4Cache")
    dev = cache.device
    if not _is(block_table, torch.int32, 2, dev):
        _check_tensor(block_table, "block_table", torch.int32, 2, dev)
    n, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table must have unit column stride")
    _check_index(seq_lens, "seq_lens", n, dev)
    if q_offsets is not None:
        _check_index(q_offsets, "q_offsets", n + 1, dev)
    elif rows != n:
        raise ValueError(f"without q_offsets there is one row per request ({rows} rows, {n} requests)")
    return dev, n, width, block_table.stride(0) if n > 1 else width


def _check_rows(t, name, heads, d, rows, dev):
    """[rows, heads, d] BF16 with unit stride along d (heads None: any); returns heads and the two strides (0 for a
    single row or head, whose stride means nothing)."""
    if not _is(t, torch.bfloat16, 3, dev):
        _check_tensor(t, name, torch.bfloat16, 3, dev)
    shape, (st, sh, sd) = t.shape, t.stride()
    if shape[2] != d or shape[0] != rows or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [{rows}, {heads}, {d}], got {tuple(shape)}")
    if sd != 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    return shape[1], st if shape[0] > 1 else 0, sh if shape[1] > 1 else 0


@_takes_stream
def nvfp4_cache_append(k, v, cache, block_table, seq_lens, q_offsets=None, with_dq=False, k_dq=None, v_dq=None):
    """Quantizes the BF16 rows k and v [tokens, heads, head_dim] into the cache.
    Request b has the rows q_offsets[b] .. q_offsets[b + 1] - 1 (one row each
    without q_offsets), its last tokens: seq_lens[b] counts them, and the pages
    come from block_table[b].  A row without a page is not stored.  With with_dq
    (or k_dq and v_dq) also returns the stored values in BF16, (k_dq, v_dq)."""
    T = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() else 0
    dev, n, width, ld = _check_requests(cache, block_table, seq_lens, q_offsets, T)
    h, d = cache.num_heads, cache.head_dim
    _, kt, kh = _check_rows(k, "k", h, d, T, dev)
    _, vt, vh = _check_rows(v, "v", h, d, T, dev)
    if with_dq or k_dq is not None or v_dq is not None:
        if k_dq is None and v_dq is None:
            k_dq, v_dq = torch.empty((2, T, h, d), dtype=torch.bfloat16, device=dev).unbind(0)
        else:
            k_dq = torch.empty((T, h, d), dtype=torch.bfloat16, device=dev) if k_dq is None else k_dq
            v_dq = torch.empty((T, h, d), dtype=torch.bfloat16, device=dev) if v_dq is None else v_dq
            for name, t in (("k_dq", k_dq), ("v_dq", v_dq)):
                _check_rows(t, name, h, d, T, dev)
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
    _launch(dev, _lib().nvfp4_cache_append, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, T, cache._ref,
            block_table.data_ptr(), ld, width, seq_lens.data_ptr(), _p(q_offsets), n, _p(k_dq), _p(v_dq))
    return (k_dq, v_dq) if k_dq is not None else None


def nvfp4_attention_workspace(tokens, q_heads, heads, head_dim, page_size, table_width, requests, ragged):
    """Bytes of workspace that nvfp4_attention needs for these shapes (ragged: with q_offsets); may be 0."""
    return _lib().nvfp4_attention_workspace(tokens, q_heads, heads, head_dim, page_size, table_width, requests,
                                            bool(ragged))


@_takes_stream
def nvfp4_attention(q, cache, block_table, seq_lens, q_offsets=None, scale=None, window=0, out=None, with_lse=False,
                    lse=None, workspace=None):
    """Causal attention of the BF16 query rows q [tokens, q_heads, head_dim]
    over the cache (requests as in nvfp4_cache_append; append their K and V
    first).  scale defaults to head_dim ** -0.5; window > 0 limits a row to
    the last `window` positions up to its own.  Returns out like q, or (out,
    lse) with with_lse (or lse): float32 [tokens, q_heads].  A row that sees
    nothing gives zeros and -inf; rows of no request are not written.
    `workspace` is a uint8 tensor of nvfp4_attention_workspace() bytes, by
    default a fresh one."""
    T = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() else 0
    dev, n, width, ld = _check_requests(cache, block_table, seq_lens, q_offsets, T)
    d = cache.head_dim
    hq, qt, qh = _check_rows(q, "q", None, d, T, dev)
    if out is None:
        out = torch.empty((T, hq, d), dtype=torch.bfloat16, device=dev)
        ot, oh = hq * d, d
    else:
        _, ot, oh = _check_rows(out, "out", hq, d, T, dev)
    if lse is None and with_lse:
        lse = torch.empty((T, hq), dtype=torch.float32, device=dev)
    elif lse is not None:
        _check_tensor(lse, "lse", torch.float32, 2, dev)
        if tuple(lse.shape) != (T, hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous [{T}, {hq}]")
    L = _lib()
    need = L.nvfp4_attention_workspace(T, hq, cache.num_heads, d, cache.page_size, width, n, q_offsets is not None)
    have = 0
    if workspace is None:
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            have = need
    else:
        _check_tensor(workspace, "workspace", torch.uint8, 1, dev)
        have = workspace.numel() if workspace.is_contiguous() else 0
    _launch(dev, L.nvfp4_attention, q.data_ptr(), qt, qh, T, hq, cache._ref, block_table.data_ptr(), ld, width,
            seq_lens.data_ptr(), _p(q_offsets), n, d ** -0.5 if scale is None else scale, window, out.data_ptr(), ot, oh,
            _p(lse), _p(workspace), have)
    return out if lse is None else (out, lse)
