"""Plain float64 references of the decode step (few-row products, the paged
NVFP4 cache, attention over it), their error bounds, and caches built from
the oracle's quantizer.  Host code only."""

import numpy as np

from oracle import formats as F, layout as OL, nvfp4 as ON

EPS_BF16, EPS_FP16, EPS_F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24   # half a step, relative


def bf16(rng, shape, scale=1.0):
    return F.bf16_rne(rng.standard_normal(shape) * scale)


class Weight:
    """One NVFP4 weight matrix [N, K] (or G of them), quantized by the oracle."""

    def __init__(self, rng, n, k, block="row", layout="linear", groups=1, std=0.02):
        self.n, self.k, self.block, self.layout = n, k, block, layout
        codes, scales, S, dq = [], [], [], []
        for _ in range(groups):
            w = F.bf16_bits_to_f64(bf16(rng, (n, k), std))
            c, s, g = (ON.quantize_tile16(w) if block == "tile" else ON.quantize_rowwise(w, "per_tensor"))
            dq.append(ON.dequantize_f64(c, s, g, "16x16" if block == "tile" else "1x16", "per_tensor"))
            scales.append(OL.linear_to_mfma(s).reshape(s.shape) if layout == "mfma" else s)
            codes.append(c)
            S.append(np.asarray(g, np.float32).reshape(1))
        self.codes, self.scales, self.S = np.stack(codes), np.stack(scales), np.concatenate(S)
        self.dq = np.stack(dq)

    def operand(self, m, torch):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        return m.Operand(m.Format.NVFP4, dev(self.codes).view(-1, self.k // 2), dev(self.scales), dev(self.S),
                         block=m.Block.TILE if self.block == "tile" else m.Block.ROW, gs=m.GScale.PER_TENSOR,
                         layout=m.Layout.MFMA if self.layout == "mfma" else m.Layout.LINEAR)


def dots(x, w):
    """x w^T in float64 and the bound of a binary32 sum of the exact products in any order
    (K additions, each a step at most: 2^-23 of the absolute sum), the factor S included."""
    y = x @ w.T
    return y, (x.shape[1] * 2 * EPS_F32 + 4 * EPS_F32) * (np.abs(x) @ np.abs(w).T)


def gemv_ref(x, w):
    y, e = dots(x, w)
    return y, EPS_BF16 * np.abs(y) + (1 + EPS_BF16) * e


def swiglu_ref(x, wg, wu):
    """silu(g) u; |silu'| <= 1.1, and sixteen binary32 roundings for exp, the quotient and the products."""
    g, eg = dots(x, wg)
    u, eu = dots(x, wu)
    silu = g / (1 + np.exp(-g))
    h = silu * u
    e = 1.1 * eg * np.abs(u) + (np.abs(silu) + 1.1 * eg) * eu + 16 * EPS_F32 * np.abs(h)
    return h, EPS_BF16 * np.abs(h) + (1 + EPS_BF16) * e


class Cache:
    """A paged cache on the host.  `fill` is the byte unused places hold (0xFF: NaN scales)."""

    def __init__(self, pages, heads, page, d, fill=0xFF):
        u8 = lambda *s: np.full(s, fill, np.uint8)
        f32 = lambda *s: np.frombuffer(np.full(int(np.prod(s)) * 4, fill, np.uint8).tobytes(), np.float32).reshape(s).copy()
        self.t = dict(k_codes=u8(pages, heads, page, d // 2), k_scales=u8(pages, heads, page, d // 16),
                      k_gscales=f32(pages, heads, page), v_codes=u8(pages, heads, page, d // 2),
                      v_scales=u8(pages, heads, d // 16, page), v_gscales=f32(pages, heads, page))
        self.pages, self.heads, self.page, self.d = pages, heads, page, d

    def put(self, name, page, slot, bits):
        """Quantizes the rows bits [heads, d] of one token (name "k" or "v"); returns their values in float64."""
        x = F.bf16_bits_to_f64(bits)
        c, s, S = ON.quantize_rowwise(x, "per_row")
        if page is not None:
            self.t[name + "_codes"][page, :, slot] = c
            if name == "k":
                self.t["k_scales"][page, :, slot] = s
            else:
                self.t["v_scales"][page, :, :, slot] = s
            self.t[name + "_gscales"][page, :, slot] = S
        return ON.dequantize_f64(c, s, S, "1x16", "per_row")

    def device(self, m, torch):
        return m.NVFP4Cache(*[torch.from_numpy(self.t[k].copy()).cuda() for k in
                              ("k_codes", "k_scales", "k_gscales", "v_codes", "v_scales", "v_gscales")])


def tables(rng, lens, page, extra=2, width_extra=0):
    """Block table of requests with `lens` tokens over shuffled pages (unused entries -1) and the page count."""
    need = [(n + page - 1) // page for n in lens]
    order = rng.permutation(sum(need) + extra)
    t = np.full((len(lens), max(need + [1]) + width_extra), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, sum(need) + extra


def attention_ref(q, k, v, pos, scale, window, seen=None):
    """One head: q [n, D], k and v [L, D] float64, pos [n].  Returns out, lse and their bounds.

    Bound: every weight p_t is off by a factor 1 + e, where e covers the logit (D binary32 additions of exact
    products, the second scale, the factor scale log2 e, the subtraction of the maximum) and the exponential.
    Weight and value meet in FP16: at most three roundings of 2^-11 (the weight; the block scale times the second
    scale, and that times the code), or 2^-25 absolute below 2^-14, where the weight 1 (one of them is at least
    that) stands for 2^10 and the largest |v| for 2688 2^3 at least: 2^-35 and 2^-38 of the largest |v| per token,
    twice that for Sref being up to twice the largest second scale.  The sums over tokens are binary32; the
    output is rounded to BF16."""
    n, L, D = q.shape[0], k.shape[0], q.shape[1]
    x = scale * (q @ k.T)
    t = np.arange(L)[None]
    ok = t <= pos[:, None]
    if window:
        ok &= t > pos[:, None] - window
    if seen is not None:
        ok &= seen[None]
    ex = scale * (D + 4) * 2 * EPS_F32 * (np.abs(q) @ np.abs(k).T) + 8 * EPS_F32 * np.abs(x)
    # q below 2^-27 of its row's largest element loses bits
    ex += scale * 2.0 ** -37 * np.abs(q).max(1, keepdims=True) * np.abs(k).sum(1)[None]
    ex = np.where(ok, ex, 0).max(1, initial=0) + 2.0 ** -20
    out, lse = np.zeros((n, D)), np.full(n, -np.inf)
    tol = np.zeros((n, D))
    for i in range(n):
        if not ok[i].any():
            continue
        xi = np.where(ok[i], x[i], -np.inf)
        top = xi.max()
        p = np.exp(xi - top)
        total = p.sum()
        p /= total
        lse[i] = top + np.log(total)
        vi = np.where(ok[i][:, None], v, 0.0)
        out[i] = p @ vi
        mass = p @ np.abs(vi)
        small = 2.0 ** -33 * ok[i].sum() * np.abs(vi).max()
        tol[i] = (EPS_BF16 * np.abs(out[i]) + (1 + EPS_BF16) * (3 * EPS_FP16 + 2 * ex[i] + 2 * EPS_F32 * (ok[i].sum() + 32))
                  * mass + small)
    lse_tol = ex + 2 * EPS_F32 * (ok.sum(1) + 32) + 4 * EPS_F32 * np.where(np.isfinite(lse), np.abs(lse), 0)
    return out, lse, tol, lse_tol
