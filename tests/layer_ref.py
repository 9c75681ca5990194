"""Plain float64 references of the steps around a layer's products (the norm,
the router and the experts' rows, rotary positions) with their error bounds.
Host code only.

Bounds count roundings: half a step of BF16 is 2^-8 of the value, of binary32
2^-24, a binary32 sum of n terms is off by at most n steps of 2^-23 of the sum
of their magnitudes in any order."""

import numpy as np

from oracle import formats as F

EPS_BF16, EPS_F32 = 2.0 ** -8, 2.0 ** -24     # half a step, relative
TINY_BF16 = 2.0 ** -134                       # half a step of the smallest BF16 values


def bf16(rng, shape, scale=1.0):
    return F.bf16_rne(rng.standard_normal(shape) * scale)


def f64(bits):
    return F.bf16_bits_to_f64(bits)


def norm_ref(x, w, eps, residual=None):
    """h (float64, BF16 values), rstd in float64, y in float64 before its rounding."""
    h = x if residual is None else f64(F.bf16_rne(x + residual))
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w


def norm_y_bits(h, rstd32, w):
    """bf16(fl(fl(h rstd) w)) in the steps of the definition, from binary32 rstd."""
    with np.errstate(all="ignore"):
        t = (h.astype(np.float32) * rstd32[:, None]).astype(np.float32)
        return F.bf16_rne((t * w.astype(np.float32)).astype(np.float32).astype(np.float64))


def norm_backward_ref(dy, h, w, rstd, dres=None):
    """dx and dw in float64 from binary32 rstd, and the bounds of the kernel's binary32 steps."""
    n = h.shape[1]
    r = rstd.astype(np.float64)[:, None]
    xhat, g = h * r, dy * w
    m = (g * xhat).mean(1, keepdims=True)
    dx = r * (g - xhat * m)
    # every term of m: xhat, t = dy xhat and its product are a rounding each, then n additions
    em = (n + 4) * 2 * EPS_F32 * np.abs(g * xhat).mean(1, keepdims=True) + 4 * EPS_F32 * np.abs(m)
    e = r * (np.abs(xhat) * em + 4 * EPS_F32 * (np.abs(g) + np.abs(xhat * m)))
    if dres is not None:
        dx = dx + dres
    e = e + 2 * EPS_F32 * np.abs(dx)
    dw = (dy * xhat).sum(0)
    ew = (h.shape[0] + 4) * 2 * EPS_F32 * np.abs(dy * xhat).sum(0)
    return dx, dw, EPS_BF16 * np.abs(dx) + (1 + EPS_BF16) * e + TINY_BF16, ew


# ------------------------------------------------------------ the experts' rows

def route_ref(x, k, renorm):
    """experts [T, k] (-1: none), weights [T, k] in float64 and their bound, from logits x [T, E] (float64).

    A weight is exp(d) over a sum, d = x - max: binary32 rounds d (d 2^-24 on the exponential), the exponential (four
    half steps), each of the n additions and the quotient."""
    T, E = x.shape
    order = np.where(np.isnan(x), np.inf, x)
    # NaN before +inf, then by value, then by index
    place = np.lexsort((np.broadcast_to(np.arange(E), x.shape), -order, ~np.isnan(x)), axis=1)[:, :k]
    top = np.take_along_axis(x, place, 1)
    chosen = ~(top == -np.inf)
    with np.errstate(all="ignore"):
        d = top - top[:, :1]
        p = np.exp(d)
        total = np.where(chosen, p, 0).sum(1) if renorm else np.exp(x - top[:, :1]).sum(1)
        w = np.where(chosen, p / total[:, None], 0.0)
        spread = np.where(chosen, np.abs(d), 0).max(1)[:, None] if renorm else np.abs(
            np.where(x > -np.inf, x - top[:, :1], 0)).max(1)[:, None]
        tol = np.where(chosen, w * (2 * spread + 2 * E + 16) * EPS_F32 + 2.0 ** -148, 0.0)
    return np.where(chosen, place, -1).astype(np.int32), w, tol


def rows_ref(ids, E):
    """offsets, row_token, row_of of ids [T, k]: rows by (expert, token, slot)."""
    T, k = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)[:E]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(offsets[-1])
    row_token, row_of = np.zeros(T * k, np.int32), np.full(T * k, -1, np.int32)
    row_token[:n] = order[:n] // k
    row_of[order[:n]] = np.arange(n)
    return offsets, row_token, row_of.reshape(T, k)


def route_backward_ref(dw, x, ids, w, renorm):
    """dlogits in float64 (weights w in float64) and a bound: w is off by its own bound, which is passed on."""
    T, E = x.shape
    has = ids >= 0
    mean = np.where(has, w * dw, 0).sum(1)[:, None]
    d = np.zeros((T, E))
    size = np.zeros((T, E))
    if not renorm:
        with np.errstate(all="ignore"):
            p = np.exp(x - x.max(1, keepdims=True))
            p = np.nan_to_num(p / p.sum(1, keepdims=True))
        d = -p * mean
        size = p * np.where(has, w * np.abs(dw), 0).sum(1)[:, None]
    for t in range(T):
        for j in range(ids.shape[1]):
            if has[t, j]:
                d[t, ids[t, j]] += w[t, j] * (dw[t, j] - mean[t, 0] if renorm else dw[t, j])
                size[t, ids[t, j]] += w[t, j] * (np.abs(dw[t, j]) + np.where(has[t], w[t] * np.abs(dw[t]), 0).sum())
    spread = np.where(np.isfinite(x), np.abs(x - x.max(1, keepdims=True)), 0).max(1, keepdims=True)
    return d, size * (4 * spread + 4 * E + 64) * EPS_F32 + 2.0 ** -140


def combine_ref(rows, row_of, weights):
    """out [T, cols] in float64 and its bound."""
    T, k = row_of.shape
    ok = (row_of >= 0) & (row_of < rows.shape[0])
    y = np.where(ok[..., None], rows[np.where(ok, row_of, 0)], 0.0)
    w = np.ones((T, k)) if weights is None else weights
    t = y * w[..., None]
    out = t.sum(1)
    e = (k + 1) * 2 * EPS_F32 * np.abs(t).sum(1)
    return out, EPS_BF16 * np.abs(out) + (1 + EPS_BF16) * e + TINY_BF16


# ------------------------------------------------------------ rotary positions

def turned_bits(bits, pos, inv_freq, interleaved, factor=1.0):
    """Rows bits [n, heads, D] (BF16) at positions pos [n] turned by the steps of the definition: BF16 bits."""
    x = f64(bits).astype(np.float32)
    rot = 2 * len(inv_freq)
    angle = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float32).astype(np.float64)
    c = (np.cos(angle) * factor).astype(np.float32)[:, None]
    s = (np.sin(angle) * factor).astype(np.float32)[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    with np.errstate(all="ignore"):
        u, v = a * c - b * s, b * c + a * s
    out = x.copy()
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2] = u, v
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = u, v
    res = F.bf16_rne(out.astype(np.float64))
    res[..., rot:] = bits[..., rot:]
    return res
