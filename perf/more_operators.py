"""The steps of a decoder layer around its quantized products, as measured cases:

    mx_rmsnorm, mx_rmsnorm_backward            residual addition, root-mean-square norm, output quantized on the way
    mx_moe_route, mx_moe_route_backward        router: the k best experts of a token, their weights, rows sorted by expert
    mx_moe_dispatch, mx_moe_combine,           tokens to their experts' rows and back with weights, and the gradients
      mx_moe_combine_backward
    nvfp4_rope_append                          rotary positions for q and k, k and v quantized into an NVFP4 cache

With `own` false, `run` computes the same operators from elementary torch operations.
Sizes: Qwen3-30B-A3B experts (hidden 2048, 128 experts, top 8, 8192 tokens), Qwen3-8B and Llama-3-8B (hidden 4096,
8192 and 32768 tokens); heads, contexts and pages are generic.
"""

import math

import torch

own = False


def listed():
    return [
        # the norm before a projection while one sequence decodes: the smallest call, latency alone
        dict(name="norm_decode_m1", op="norm", rows=1, cols=4096, fmt="bf16", layout="linear", residual=True, rstd=False),
        # a learner's norm with its residual, MXFP8 for the next product, the stored values for the backward (Qwen3-8B)
        dict(name="norm_mxfp8_t8192", op="norm", rows=8192, cols=4096, fmt="mxfp8", layout="mfma", residual=True, rstd=True),
        # the same with NVFP4 per token, a ragged number of tokens (Llama-3-8B)
        dict(name="norm_nvfp4_t32001", op="norm", rows=32001, cols=4096, fmt="nvfp4", layout="linear", residual=True,
             rstd=True),
        # the gradient of an odd, short batch (Qwen3-30B-A3B)
        dict(name="norm_bwd_t1003", op="norm_bwd", rows=1003, cols=2048, residual=False),
        # a learner's gradient with the residual stream's (Llama-3-8B)
        dict(name="norm_bwd_t32768", op="norm_bwd", rows=32768, cols=4096, residual=True),
        # 64 sequences decode: router to sorted rows, a chain of latencies
        dict(name="route_decode_t64", op="route", t=64, e=128, k=8, dtype="f32", renorm=True, masked=0.0, train=False),
        # a learner's batch, the gradient of the logits with it
        dict(name="route_train_t8192", op="route", t=8192, e=128, k=8, dtype="f32", renorm=False, masked=0.0, train=True),
        # 64 sequences decode: the experts' rows weighted and summed
        dict(name="moe_decode_t64", op="moe", t=64, e=128, k=8, h=2048, dropped=0.0, train="decode"),
        # a learner's batch: tokens to rows, rows back to tokens
        dict(name="moe_forward_t8192", op="moe", t=8192, e=128, k=8, h=2048, dropped=0.0, train="forward"),
        # its gradients; a quarter of the experts is on another device
        dict(name="moe_backward_t8192", op="moe", t=8192, e=128, k=8, h=2048, dropped=0.25, train="backward"),
        # one decode step of 128 sequences
        dict(name="rope_append_b128", op="rope", b=128, ctx=2000, q=1, hq=32, hkv=8, d=128, rot=128, page=16, pairs="half",
             scaled=False),
        # three prompts behind long contexts, scaled positions
        dict(name="rope_append_prompts", op="rope", b=3, ctx=40000, q=4001, hq=32, hkv=8, d=128, rot=128, page=64,
             pairs="half", scaled=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "route", "moe", "moe", "rope", "rope"])
    if op in ("norm", "norm_bwd"):
        unit = {"norm": 128, "norm_bwd": 8}[op]
        cols = unit * _log(rng, 1, 16384 // unit)
        rows = _log(rng, 1, min(40000, 80_000_000 // cols))
        case = dict(op=op, rows=rows, cols=cols, residual=rng.choice([False, True]))
        if op == "norm":
            case["fmt"] = rng.choice(["bf16", "mxfp8", "nvfp4", "fp8_b128", "fp8_b128_f32"])
            case["layout"] = rng.choice(["linear", "mfma"]) if case["fmt"] in ("mxfp8", "nvfp4") else "linear"
            case["rstd"] = rng.choice([False, True])
            if case["layout"] == "mfma":
                case["rows"] = (rows + 31) // 32 * 32
        return case
    if op == "route":
        e = _log(rng, 4, 512)
        return dict(op=op, t=_log(rng, 1, 8192), e=e, k=rng.randrange(1, min(e, 8) + 1), dtype=rng.choice(["f32", "bf16"]),
                    renorm=rng.choice([False, True]), masked=rng.choice([0.0, 0.0, 0.3]), train=rng.choice([False, True]))
    if op == "moe":
        e = _log(rng, 4, 256)
        k = rng.randrange(1, min(e, 8) + 1)
        h = 8 * _log(rng, 8, 900)
        return dict(op=op, t=_log(rng, 1, min(12000, 100_000_000 // (k * h))), e=e, k=k, h=h,
                    dropped=rng.choice([0.0, 0.0, 0.5]), train=rng.choice(["decode", "forward", "backward"]))
    d = rng.choice([64, 128, 128, 256])
    q = rng.choice([1, 1, _log(rng, 2, 2000)])
    hkv = rng.choice([1, 2, 4, 8])
    return dict(op=op, b=_log(rng, 1, 200 if q == 1 else 4), ctx=q + _log(rng, 1, 20000 if q > 1 else 2000), q=q,
                hq=hkv * rng.choice([1, 2, 3, 4, 8]), hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4]),
                page=rng.choice([16, 32, 64, 128]), pairs=rng.choice(["half", "interleaved"]),
                scaled=rng.choice([False, True]))


_CODE_BYTES = {"bf16": 2, "mxfp8": 3 + 1 / 32, "nvfp4": 2.5 + 1 / 16, "fp8_b128": 3 + 1 / 128, "fp8_b128_f32": 3 + 1 / 32}


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["cols"]
        each = 2 + _CODE_BYTES[case["fmt"]] + (4 if case["residual"] else 0)
        per_row = (4 if case["rstd"] else 0) + (4 if case["fmt"] == "nvfp4" else 0)
        return {"bytes": n * each + case["rows"] * per_row + 2 * case["cols"], "flops": 6 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (8 if case["residual"] else 6) + 4 * case["rows"] + 6 * case["cols"], "flops": 9 * n}
    if op == "route":
        t, e, k, w = case["t"], case["e"], case["k"], 4 if case["dtype"] == "f32" else 2
        ints = 4 * (4 * t * k + e + 1)
        return {"bytes": t * e * w + ints + ((0 if case["renorm"] else t * e * w) + t * e * w + 12 * t * k
                                             if case["train"] else 0), "flops": 4 * t * e}
    if op == "moe":
        t, k, h = case["t"], case["k"], case["h"]
        rows = t * k * (1 - case["dropped"])
        one, all_ = 2 * t * h, 2 * rows * h                               # tokens, experts' rows
        if case["train"] == "decode":
            return {"bytes": one + all_ + 8 * t * k, "flops": 2 * rows * h}
        if case["train"] == "forward":
            return {"bytes": 2 * one + 2 * all_ + 12 * t * k, "flops": 2 * rows * h}
        # dout and rows read, drows and dweights written; then the experts' input gradients back to the tokens
        return {"bytes": one + 2 * all_ + 12 * t * k + all_ + one + 4 * t * k, "flops": 4 * rows * h}
    d, row = case["d"], case["d"] // 2 + case["d"] // 16 + 4
    tokens = sum(q for _, q in _lengths(case))
    return {"bytes": tokens * (4 * case["hq"] * d + 2 * case["hkv"] * (4 * d + row)),
            "flops": tokens * (3 * case["hq"] * case["rot"] + case["hkv"] * (3 * case["rot"] + 4 * d))}


def _lengths(case):
    """(context, new tokens) of every request: ragged, the first one the longest.  The context counts the new tokens."""
    out = []
    for i in range(case["b"]):
        q = 1 + int((case["q"] - 1) * (1 - 0.5 * ((i * 0.382) % 1)))
        out.append((max(q, int(case["ctx"] * (1 - 0.9 * ((i * 0.618) % 1)))), q))
    return out


# ------------------------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "norm_bwd": _prepare_norm, "route": _prepare_route, "moe": _prepare_moe,
            "rope": _prepare_rope}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


_EPS = 1e-6


def _prepare_norm(case, g):
    rows, cols = case["rows"], case["cols"]
    bf16 = torch.bfloat16
    loud = torch.exp(_randn(g, rows, 1))                                  # a magnitude per token
    st = dict(case=case, w=(1 + 0.1 * _randn(g, cols)).to(bf16), x=(_randn(g, rows, cols) * loud).to(bf16))
    st["r"] = _randn(g, rows, cols).to(bf16) if case["residual"] else None
    if case["op"] == "norm_bwd":
        st["h"] = st.pop("x")
        st["dy"] = (_randn(g, rows, cols) * 1e-3).to(bf16)
        st["rstd"] = (1 / torch.sqrt(st["h"].double().square().mean(1) + _EPS)).float()
        if case["residual"]:
            st["r"] = (st["r"].float() * 1e-3).to(bf16)                   # the gradient that the residual stream brings
    return st


def _prepare_route(case, g):
    t, e, k = case["t"], case["e"], case["k"]
    logits = _randn(g, t, e)
    if case["masked"]:                                                    # experts that a token may not use
        hide = torch.rand(t, e, generator=g, device="cuda") < case["masked"]
        logits = logits.masked_fill(hide, -math.inf)
    if case["dtype"] == "bf16":
        logits = logits.to(torch.bfloat16)
    st = dict(case=case, logits=logits)
    if case["train"]:
        st["dweights"] = _randn(g, t, k) * 1e-3
    return st


def _prepare_moe(case, g):
    t, e, k, h = case["t"], case["e"], case["k"], case["h"]
    bf16 = torch.bfloat16
    ids = _randn(g, t, e).topk(k, dim=1).indices
    if case["dropped"]:                                                   # the first experts are here, the others elsewhere
        ids = torch.where(ids < max(1, round(e * (1 - case["dropped"]))), ids, torch.full_like(ids, -1))
    row_of = _sorted_rows(ids.int(), e)[2]
    st = dict(case=case, row_of=row_of, weights=torch.softmax(_randn(g, t, k), 1))
    rows = lambda s: (_randn(g, t * k, h) * s).to(bf16)
    if case["train"] == "forward":
        st["x"] = _randn(g, t, h).to(bf16)
    if case["train"] != "backward":
        st["rows"] = rows(1)
    else:
        st["rows"], st["dx_rows"] = rows(1), rows(1e-3)
        st["dout"] = (_randn(g, t, h) * 1e-3).to(bf16)
    if case["train"] != "decode":
        st["out"] = torch.zeros((t * k, h), dtype=bf16, device="cuda")    # rows of no expert stay as they are
    return st


_CACHE = ("k_codes", "k_scales", "k_gscales", "v_codes", "v_scales", "v_gscales")


def _prepare_rope(case, g):
    b, h, d, p, rot = case["b"], case["hkv"], case["d"], case["page"], case["rot"]
    lens = _lengths(case)
    need = [(c + p - 1) // p for c, _ in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()       # pages of a running server: no order
    table = torch.full((b, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    f32 = lambda *s: torch.zeros(s, dtype=torch.float32, device="cuda")
    offs = [0]
    for _, q in lens:
        offs.append(offs[-1] + q)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if case["scaled"]:                                                    # slow pairs stretched by 8, fast ones kept
        keep = ((inv * 4096 / (2 * math.pi) - 1) / 31).clamp(0, 1)
        inv = inv * keep + inv / 8 * (1 - keep)
    channel = torch.exp(0.5 * _randn(g, h, d))                            # keys have loud channels
    st = dict(case=case, table=table, seq_lens=torch.tensor([c for c, _ in lens], dtype=torch.int32, device="cuda"),
              q_offsets=None if case["q"] == 1 else torch.tensor(offs, dtype=torch.int32, device="cuda"),
              inv_freq=inv.float(), factor=0.1 * math.log(8) + 1 if case["scaled"] else 1.0,
              q=_randn(g, offs[-1], case["hq"], d).to(torch.bfloat16),
              k=(_randn(g, offs[-1], h, d) * channel).to(torch.bfloat16), v=_randn(g, offs[-1], h, d).to(torch.bfloat16),
              k_codes=u8(pages, h, p, d // 2), k_scales=u8(pages, h, p, d // 16), k_gscales=f32(pages, h, p),
              v_codes=u8(pages, h, p, d // 2), v_scales=u8(pages, h, d // 16, p), v_gscales=f32(pages, h, p))
    if own:
        import microscaling_quantization_block_amd as mxq
        st["cache"] = mxq.NVFP4Cache(*[st[c] for c in _CACHE])
    return st


# ---------------------------------------------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "route": _plain_route, "moe": _plain_moe,
            "rope": _plain_rope}[op](state)


def _own(op, st):
    import microscaling_quantization_block_amd as mxq
    case = st["case"]
    if op == "norm":
        fmt = mxq.Format[case["fmt"].upper()]
        n = mxq.mx_rmsnorm(st["x"], st["w"], _EPS, residual=st["r"], fmt=fmt, layout=mxq.Layout[case["layout"].upper()],
                           with_dq=fmt != mxq.Format.BF16, with_rstd=case["rstd"])
        return dict(h=n.h, y=n.y if fmt == mxq.Format.BF16 else n.dq, rstd=n.rstd)
    if op == "norm_bwd":
        dx, dw = mxq.mx_rmsnorm_backward(st["dy"], st["h"], st["w"], st["rstd"], dresidual=st["r"])
        return dict(dx=dx, dw=dw)
    if op == "route":
        r = mxq.mx_moe_route(st["logits"], case["k"], renormalize=case["renorm"])
        out = r._asdict()
        if case["train"]:
            out["dlogits"] = mxq.mx_moe_route_backward(st["dweights"], st["logits"], r.experts, r.weights,
                                                       renormalize=case["renorm"])
        return out
    if op == "moe":
        if case["train"] == "decode":
            return mxq.mx_moe_combine(st["rows"], st["row_of"], st["weights"])
        if case["train"] == "forward":
            rows = mxq.mx_moe_dispatch(st["x"], st["row_of"], out=st["out"])
            return rows, mxq.mx_moe_combine(st["rows"], st["row_of"], st["weights"])
        drows, dw = mxq.mx_moe_combine_backward(st["dout"], st["rows"], st["row_of"], st["weights"], drows=st["out"])
        return drows, dw, mxq.mx_moe_combine(st["dx_rows"], st["row_of"])
    q, k, v = mxq.nvfp4_rope_append(st["q"], st["k"], st["v"], st["cache"], st["table"], st["seq_lens"], st["inv_freq"],
                                    q_offsets=st["q_offsets"], interleaved=case["pairs"] == "interleaved",
                                    factor=st["factor"], with_dq=True)
    return dict(q=q, k=k, v=v, **{c: st[c] for c in _CACHE})


# The norm.  The quantized output is held to the steps of the formats, so the statistics are taken in 64 bits and
# every other step is one binary32 operation: a sum in another order would move values over the borders of codes.

def _plain_norm(st):
    case = st["case"]
    h = st["x"] if st["r"] is None else (st["x"].float() + st["r"].float()).to(torch.bfloat16)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + _EPS)).float()
    y = (h.float() * rstd[:, None] * st["w"].float()).to(torch.bfloat16)
    if case["fmt"] != "bf16":
        y = {"mxfp8": _mxfp8, "nvfp4": _nvfp4, "fp8_b128": _fp8_b128, "fp8_b128_f32": _fp8_b128_f32}[case["fmt"]](y)
    return dict(h=h if st["r"] is not None else None, y=y, rstd=rstd if case["rstd"] else None)


def _pow2_blocks(y, n):
    """E4M3 codes under a power of two per block of n values: the values that they stand for."""
    yb = y.float().unflatten(-1, (-1, n))
    amax = yb.abs().amax(-1, keepdim=True)
    man, ex = torch.frexp(amax)                                           # amax = man 2^ex, man in [0.5, 1)
    e = (ex - 9 + (man > 0.875).int()).clamp(-127, 127)                   # 448 = 0.875 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    c = torch.ldexp(yb, -e).to(torch.float8_e4m3fn)
    return torch.ldexp(c.float(), e).flatten(-2).to(torch.bfloat16)


def _mxfp8(y):
    return _pow2_blocks(y, 32)


def _fp8_b128(y):
    return _pow2_blocks(y, 128)


def _fp8_b128_f32(y):
    yb = y.float().unflatten(-1, (-1, 128))
    s = yb.abs().amax(-1, keepdim=True) / 448.0
    c = torch.where(s > 0, yb / s, torch.zeros_like(yb)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (c.float() * s).flatten(-2).to(torch.bfloat16)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nvfp4_parts(x):
    """Rows of x to E2M1 codes (one a byte), E4M3 block scales (float8), S, and the BF16 values they stand for."""
    x = x.float()
    S = (x.abs().amax(-1).double() / 2688.0).float()
    xb = x.unflatten(-1, (-1, 16))
    Sb = S[..., None]
    t = (xb.abs().amax(-1).double() / (6.0 * Sb).double()).float()
    sb = torch.where(Sb > 0, t, torch.zeros_like(t)).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = sb.float() * Sb
    r = torch.where(den > 0, (1.0 / den.double()).float(), torch.zeros_like(den))
    y = xb * r[..., None]
    a = y.abs()
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    lut = torch.tensor(_E2M1, device=x.device)
    val = torch.copysign(lut[c.int()], y) * sb.float()[..., None] * Sb[..., None]
    c = (c + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return c, sb, S, val.flatten(-2).to(torch.bfloat16)


def _nvfp4(y):
    return _nvfp4_parts(y)[3]


def _plain_norm_bwd(st):
    dy, h, w, rstd = st["dy"].float(), st["h"].float(), st["w"].float(), st["rstd"][:, None]
    xhat, g = h * rstd, dy * w
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if st["r"] is not None:
        dx = dx + st["r"].float()
    return dict(dx=dx.to(torch.bfloat16), dw=(dy * xhat).double().sum(0).float())


# The router and the experts' rows.

def _sorted_rows(ids, e):
    """offsets [e + 1], the token of every row and the row of every (token, slot), rows ordered by (expert, token).
    An id of -1 has no row (-1); rows behind the last one hold token 0."""
    t, k = ids.shape
    flat = ids.flatten().long()
    key = torch.where(flat < 0, torch.full_like(flat, e), flat)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(e + 1, device=ids.device)).int()
    row_token = torch.where(key < e, order // k, torch.zeros_like(order)).int()
    row = torch.empty_like(flat)
    row[order] = torch.arange(t * k, device=ids.device)
    return offsets, row_token, torch.where(flat < 0, torch.full_like(row, -1), row).int().view(t, k)


def _plain_route(st):
    case, x = st["case"], st["logits"].float()
    k = case["k"]
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    chosen = top > -math.inf
    m = x.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    total = torch.exp(top - m).sum(1, keepdim=True) if case["renorm"] else p.sum(1, keepdim=True)
    weights = torch.where(chosen, torch.exp(top - m) / total, torch.zeros_like(top))
    experts = torch.where(chosen, ids, torch.full_like(ids, -1)).int()
    offsets, row_token, row_of = _sorted_rows(experts, case["e"])
    out = dict(experts=experts, weights=weights, offsets=offsets, row_token=row_token, row_of=row_of)
    if case["train"]:
        dw = torch.where(chosen, st["dweights"], torch.zeros_like(top))
        mean = (weights * dw).sum(1, keepdim=True)
        if case["renorm"]:
            d = torch.zeros_like(x)
        else:
            d = -(p / total.clamp(min=1e-30)) * mean
        own_part = weights * (dw - mean) if case["renorm"] else weights * dw
        out["dlogits"] = d.scatter_add(1, ids, own_part).to(st["logits"].dtype)
    return out


def _gathered(rows, row_of):
    """rows[row_of] in binary32, zeros where there is no row: [t, k, h]."""
    y = rows[row_of.clamp(min=0).long()].float()
    return y.masked_fill((row_of < 0)[..., None], 0.0)


def _to_rows(out, x, row_of):
    """x [t, k, h] to its rows of out; the others stay."""
    has = row_of >= 0
    out[row_of[has].long()] = x[has].to(out.dtype)
    return out


def _plain_moe(st):
    case, row_of = st["case"], st["row_of"]
    k = case["k"]
    w = torch.where(row_of >= 0, st["weights"], torch.zeros_like(st["weights"]))
    if case["train"] == "backward":
        dout = st["dout"].float()
        dw = (_gathered(st["rows"], row_of) * dout[:, None]).sum(-1)
        drows = _to_rows(st["out"], dout[:, None] * w[..., None], row_of)
        return drows, dw, _gathered(st["dx_rows"], row_of).sum(1).to(torch.bfloat16)
    y = (_gathered(st["rows"], row_of) * w[..., None]).sum(1).to(torch.bfloat16)
    if case["train"] == "decode":
        return y
    return _to_rows(st["out"], st["x"][:, None].expand(-1, k, -1), row_of), y


# Positions and the cache.

def _positions(st):
    """Request and position of every row."""
    row = torch.arange(st["q"].shape[0], device="cuda")
    if st["q_offsets"] is None:
        return row, (st["seq_lens"] - 1).long()
    req = torch.searchsorted(st["q_offsets"].long(), row, right=True) - 1
    return req, (st["seq_lens"][req] - st["q_offsets"][req + 1] + row).long()


def _rotate(x, cos, sin, case):
    """The first `rot` values of every head turned by the row's angles, rounded to BF16."""
    rot = case["rot"]
    y = x.float()
    c, s = cos[:, None], sin[:, None]
    if case["pairs"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(torch.bfloat16)


def _plain_rope(st):
    case = st["case"]
    req, pos = _positions(st)
    angle = pos.double()[:, None] * st["inv_freq"].double()               # far positions: 64 bits
    cos, sin = (torch.cos(angle) * st["factor"]).float(), (torch.sin(angle) * st["factor"]).float()
    out = dict(q=_rotate(st["q"], cos, sin, case))
    p = case["page"]
    page, slot = st["table"][req, pos // p].long(), pos % p
    for name, x in (("k", _rotate(st["k"], cos, sin, case)), ("v", st["v"])):
        c, s, S, out[name] = _nvfp4_parts(x)
        st[name + "_codes"][page, :, slot] = c[..., 0::2] | (c[..., 1::2] << 4)
        if name == "k":
            st["k_scales"][page, :, slot] = s.view(torch.uint8)
        else:
            st["v_scales"][page, :, :, slot] = s.view(torch.uint8)
        st[name + "_gscales"][page, :, slot] = S
    return dict(out, **{c: st[c] for c in _CACHE})


# ------------------------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "route": _exact_route, "moe": _exact_moe,
            "rope": _exact_rope}[case["op"]](case, st)


def _near(x, bits, lowest):
    """x in 64 bits rounded to `bits` significant bits, half to even, exponents from `lowest` on."""
    ulp = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** lowest))) - (bits - 1))
    return torch.round(x / ulp) * ulp


def _bf16_64(x):
    return _near(x, 8, -126)


def _fl(x):
    return x.float().double()


def _exact_quantized(y, fmt):
    """The values that the codes of rows y (64 bits, BF16 values) stand for."""
    if fmt == "nvfp4":
        # a chain of binary32 steps, each taken in 64 bits and rounded to 32
        S = _fl(y.abs().amax(-1, keepdim=True) / 2688)[..., None]
        yb = y.view(*y.shape[:-1], -1, 16)
        t = _fl(yb.abs().amax(-1, keepdim=True) / _fl(6 * S)).nan_to_num(0.0).clamp(max=448)
        sb = _near(t, 4, -6)
        z = torch.where(sb > 0, _fl(yb * _fl(1 / _fl(sb * S))), torch.zeros_like(yb))
        a = z.abs().clamp(max=6)
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = torch.round(a / step) * step
        return (_fl(_fl(q * sb) * S) * torch.where(torch.signbit(z), -1.0, 1.0)).view(y.shape)
    n = 32 if fmt == "mxfp8" else 128
    yb = y.view(*y.shape[:-1], -1, n)
    amax = yb.abs().amax(-1, keepdim=True)
    if fmt == "fp8_b128_f32":
        s = _fl(amax / 448)
        z = torch.where(s > 0, _fl(yb / s), torch.zeros_like(yb))
    else:
        s = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(-127, 127))
        z = yb / s
    return (_near(z, 4, -6).clamp(-448, 448) * s).view(y.shape)


def _exact_norm(case, st):
    h = st["x"].double()
    if st["r"] is not None:
        h = _bf16_64(h + st["r"].double())
    rstd = torch.rsqrt((h * h).sum(1) / case["cols"] + _EPS)
    y = h * rstd[:, None] * st["w"].double()
    if case["fmt"] != "bf16":
        y = _exact_quantized(_bf16_64(y), case["fmt"])
    return dict(h=None if st["r"] is None else h, y=y, rstd=rstd if case["rstd"] else None)


def _exact_norm_bwd(case, st):
    # y_i = w_i h_i (sum_j h_j^2 / n + eps)^(-1/2), differentiated: rstd is the forward's
    h, r, n = st["h"].double(), st["rstd"].double()[:, None], case["cols"]
    dy = st["dy"].double()
    dot = torch.matmul((dy * h), st["w"].double()[:, None])
    dx = r * st["w"].double() * dy - r ** 3 / n * dot * h
    if st["r"] is not None:
        dx = dx + st["r"].double()
    return dict(dx=dx, dw=torch.matmul(r.t(), dy * h)[0])


def _exact_route(case, st):
    x = st["logits"].double()
    e, k = case["e"], case["k"]
    # the place of an expert: how many are larger, or equal with a lower id
    place = torch.zeros(x.shape, dtype=torch.int64, device="cuda")
    low = torch.arange(e, device="cuda")
    for j in range(e):
        xj = x[:, j:j + 1]
        place += (xj > x) | ((xj == x) & (j < low))
    live = x > -math.inf
    pick = (place < k) & live
    mass = torch.exp(x - x.amax(1, keepdim=True)).nan_to_num(0.0)
    total = torch.where(pick, mass, torch.zeros_like(mass)).sum(1, keepdim=True) if case["renorm"] else mass.sum(1, keepdim=True)
    p = (mass / total).nan_to_num(0.0)
    slot = torch.where(pick, place, torch.full_like(place, k))
    weights = torch.zeros(x.shape[0], k + 1, dtype=torch.float64, device="cuda").scatter(1, slot, p)[:, :k]
    out = dict(experts=None, weights=weights, offsets=None, row_token=None, row_of=None)
    if case["train"]:
        # dw of every expert (0 where it was not chosen); softmax over the chosen, or over all
        dw = torch.cat([st["dweights"].double(), torch.zeros_like(x[:, :1])], 1).gather(1, slot)
        base = torch.where(pick, p, torch.zeros_like(p)) if case["renorm"] else p
        out["dlogits"] = base * (dw - (p * dw).sum(1, keepdim=True))
    return out


def _exact_moe(case, st):
    t, k, h = case["t"], case["k"], case["h"]
    row_of = st["row_of"].long()

    def combined(rows, weights):
        y = torch.zeros(t, h, dtype=torch.float64, device="cuda")
        for j in range(k):
            has = row_of[:, j] >= 0
            y[has] += weights[has, j, None] * rows[row_of[has, j]].double()
        return y

    w = st["weights"].double()
    if case["train"] == "decode":
        return combined(st["rows"], w)
    out = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
    if case["train"] == "forward":
        for j in range(k):
            has = row_of[:, j] >= 0
            out[row_of[has, j]] = st["x"][has].double()
        return out, combined(st["rows"], w)
    dout, dw = st["dout"].double(), torch.zeros_like(w)
    for j in range(k):
        has = row_of[:, j] >= 0
        at = row_of[has, j]
        out[at] = w[has, j, None] * dout[has]
        dw[has, j] = (st["rows"][at].double() * dout[has]).sum(1)
    return out, dw, combined(st["dx_rows"], torch.ones_like(w))


def _exact_rope(case, st):
    rot, d = case["rot"], case["d"]
    pos = torch.cat([torch.arange(c - q, c, device="cuda") for c, q in _lengths(case)]).double()
    i = torch.arange(rot // 2, device="cuda")
    one, two = (i, i + rot // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
    turn = torch.polar(torch.full((pos.numel(), rot // 2), st["factor"], dtype=torch.float64, device="cuda"),
                       pos[:, None] * st["inv_freq"].double())[:, None]

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., one], y[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
        return y

    return dict(q=turned(st["q"]), k=_exact_quantized(_bf16_64(turned(st["k"])), "nvfp4"),
                v=_exact_quantized(st["v"].double(), "nvfp4"), **{c: None for c in _CACHE})
