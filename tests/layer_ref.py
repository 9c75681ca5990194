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
