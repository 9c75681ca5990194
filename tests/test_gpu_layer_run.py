"""A decoder layer with experts on this library alone: norm, projections, rotated append, attention, norm, router,
experts' products, their sum.  Stage by stage against float64 on the stage's own input; the step captured into a graph;
and the learner's gradients of the norm, the router and the experts' rows in one chain."""

import numpy as np
import pytest
import torch

from oracle import formats as F, nvfp4 as ON
from tests import decode_ref as D, layer_ref as R
from tests.util import from_dev_bf16, requires_gpu, say, to_dev_bf16, to_np

pytestmark = [pytest.mark.gpu, requires_gpu]

HID, HQ, HKV, HD, INTER, E, K, PAGE, EPS = 256, 4, 2, 64, 192, 16, 3, 16, 1e-6
CACHE = ("k_codes", "k_scales", "k_gscales", "v_codes", "v_scales", "v_gscales")


def _m():
    import microscaling_quantization_block_amd as m
    return m


def _f64(t):
    return R.f64(from_dev_bf16(t))


class Layer:
    def __init__(self, seed, lens, pages=60, width=10):
        rng = np.random.default_rng(seed)
        m = _m()
        self.w = dict(qkv=D.Weight(rng, (HQ + 2 * HKV) * HD, HID), o=D.Weight(rng, HID, HQ * HD, block="tile"),
                      router=D.Weight(rng, E, HID, std=0.2), gate_up=D.Weight(rng, 2 * INTER, HID, groups=E),
                      down=D.Weight(rng, HID, INTER, groups=E))
        self.op = {k: w.operand(m, torch) for k, w in self.w.items()}
        self.norm = [F.bf16_rne(1 + 0.1 * rng.standard_normal(HID)) for _ in range(2)]
        self.norm_d = [to_dev_bf16(w) for w in self.norm]
        self.freq = (10000.0 ** (-np.arange(0, HD, 2) / HD)).astype(np.float32)
        self.freq_d = torch.from_numpy(self.freq).cuda()
        self.b = len(lens)
        self.table = torch.from_numpy(rng.permutation(pages)[:self.b * width].reshape(self.b, width).astype(np.int32)).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cache = m.NVFP4Cache.empty(pages, HKV, PAGE, HD)
        for n in CACHE:
            getattr(self.cache, n).view(torch.uint8).fill_(0xFF)          # stale pages
        n = [x - 1 for x in lens]                                         # the prompts: all but the first decoded token
        offs = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device="cuda")
        q, k, v = (to_dev_bf16(R.bf16(rng, (sum(n), h, HD))) for h in (HQ, HKV, HKV))
        m.nvfp4_rope_append(q, k, v, self.cache, self.table, self.lens - 1, self.freq_d, q_offsets=offs)
        self.x, self.r = (to_dev_bf16(R.bf16(rng, (self.b, HID))) for _ in range(2))

    def step(self, x, r):
        """The layer's output and residual stream; also every stage's result."""
        m, b = _m(), self.b
        n1 = m.mx_rmsnorm(x, self.norm_d[0], EPS, residual=r, with_rstd=True)
        qkv = m.nvfp4_gemv(n1.y, self.op["qkv"], b, (HQ + 2 * HKV) * HD, HID).view(b, -1, HD)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        qr = m.nvfp4_rope_append(q, k, v, self.cache, self.table, self.lens, self.freq_d)
        att = m.nvfp4_attention(qr, self.cache, self.table, self.lens)
        o = m.nvfp4_gemv(att.view(b, -1), self.op["o"], b, HID, HQ * HD)
        n2 = m.mx_rmsnorm(o, self.norm_d[1], EPS, residual=n1.h, with_rstd=True)
        logits = m.nvfp4_gemv(n2.y, self.op["router"], b, E, HID)
        rt = m.mx_moe_route(logits, K)
        hh = m.nvfp4_gemv_swiglu(n2.y, self.op["gate_up"], b * K, INTER, HID, group_row_offsets=rt.offsets,
                                 x_row_index=rt.row_token)
        dn = m.nvfp4_gemv(hh, self.op["down"], b * K, HID, INTER, group_row_offsets=rt.offsets)
        out = m.mx_moe_combine(dn, rt.row_of, rt.weights)
        return out, n2.h, dict(x=x, r=r, n1=n1, qkv=qkv, qr=qr, att=att, o=o, n2=n2, logits=logits, rt=rt, hh=hh, dn=dn)


def _cached(s, name, b, ctx):
    codes, scales, gs = (getattr(s.cache, f"{name}_{n}").cpu().numpy() for n in ("codes", "scales", "gscales"))
    table, out = s.table.cpu().numpy(), np.zeros((HKV, ctx, HD))
    for t in range(ctx):
        p, slot = table[b, t // PAGE], t % PAGE
        sc = scales[p, :, slot] if name == "k" else scales[p, :, :, slot]
        out[:, t] = ON.dequantize_f64(codes[p, :, slot], sc, gs[p, :, slot], "1x16", "per_row")
    return out


def _check_norm(n, x, w, r):
    h, rstd, _ = R.norm_ref(x, R.f64(w), EPS, r)
    assert np.array_equal(_f64(n.h), h)
    assert (np.abs(to_np(n.rstd) - rstd) <= (R.EPS_F32 + 2.0 ** -40) * rstd).all()
    assert np.array_equal(from_dev_bf16(n.y), R.norm_y_bits(h, to_np(n.rstd), R.f64(w)))


def test_steps_stage_by_stage():
    s = Layer(1, [1, 17, 40, 100, 5])
    x, r = s.x, s.r
    for i in range(3):
        say(f"layer step {i}")
        nx, nr, st = s.step(x, r)
        lens = s.lens.cpu().numpy()
        _check_norm(st["n1"], _f64(st["x"]), s.norm[0], _f64(st["r"]))
        _check_norm(st["n2"], _f64(st["o"]), s.norm[1], _f64(st["n1"].h))
        for name, a, w in (("qkv", st["n1"].y, "qkv"), ("o", st["att"].view(s.b, -1), "o"), ("logits", st["n2"].y, "router")):
            ref, tol = D.gemv_ref(_f64(a), s.w[w].dq[0])
            assert (np.abs(_f64(st[name]).reshape(s.b, -1) - ref) <= tol).all(), (i, name)
        qkv = from_dev_bf16(st["qkv"])
        assert np.array_equal(from_dev_bf16(st["qr"]), R.turned_bits(qkv[:, :HQ], lens - 1, s.freq, False))
        kt = R.turned_bits(qkv[:, HQ:HQ + HKV], lens - 1, s.freq, False)
        q, att = _f64(st["qr"]), _f64(st["att"])
        for b in range(s.b):
            k, v = _cached(s, "k", b, lens[b]), _cached(s, "v", b, lens[b])
            c, sc, S = ON.quantize_rowwise(R.f64(kt[b]), "per_row")
            assert np.array_equal(k[:, -1], ON.dequantize_f64(c, sc, S, "1x16", "per_row"))
            for h in range(HQ):
                o, _, tol, _ = D.attention_ref(q[b:b + 1, h], k[h // 2], v[h // 2], lens[b:b + 1] - 1, HD ** -0.5, 0)
                assert (np.abs(att[b, h] - o[0]) <= tol[0]).all(), (i, b, h)
        rt = st["rt"]
        ids, w, tol = R.route_ref(_f64(st["logits"]), K, True)
        assert np.array_equal(to_np(rt.experts), ids) and (np.abs(to_np(rt.weights) - w) <= tol).all()
        off, tok, row_of = R.rows_ref(ids, E)
        assert all(np.array_equal(to_np(a), b) for a, b in zip(rt[2:], (off, tok, row_of)))
        y, hh, dn = _f64(st["n2"].y), _f64(st["hh"]), _f64(st["dn"])
        for e in range(E):
            rows = slice(off[e], off[e + 1])
            gu = s.w["gate_up"].dq[e]
            ref, tol = D.swiglu_ref(y[tok[rows]], gu[:INTER], gu[INTER:])
            assert (np.abs(hh[rows] - ref) <= tol).all(), (i, e)
            ref, tol = D.gemv_ref(hh[rows], s.w["down"].dq[e])
            assert (np.abs(dn[rows] - ref) <= tol).all(), (i, e)
        ref, tol = R.combine_ref(dn, row_of, to_np(rt.weights).astype(np.float64))
        assert (np.abs(_f64(nx) - ref) <= tol).all(), i
        x, r = nx, nr
        s.lens += 1


def test_captured_step():
    """A captured step advances the lengths itself; each replay equals the eager step, bit for bit, with eager work of the
    program between the replays."""
    lens = [5, 60, 31]
    eager, s = Layer(2, lens), Layer(2, lens)
    xb, rb = s.x.clone(), s.r.clone()
    say("capture layer")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step(xb, rb)                                     # warm up; writes the token that the first replay rewrites
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x, r, _ = s.step(xb, rb)
        xb.copy_(x)
        rb.copy_(r)
        s.lens.add_(1)
    x, r = eager.x, eager.r
    for i in range(5):
        say(f"replay layer {i}")
        g.replay()
        x, r, _ = eager.step(x, r)
        eager.lens += 1
        torch.cuda.synchronize()
        assert torch.equal(xb, x) and torch.equal(rb, r), i
        assert torch.equal(s.cache.k_codes, eager.cache.k_codes) and torch.equal(s.cache.v_scales, eager.cache.v_scales)


@pytest.mark.parametrize("fmt,layout", [("NVFP4", "MFMA"), ("NVFP4", "LINEAR"), ("MXFP8", "MFMA")])
def test_norm_feeds_the_products(fmt, layout):
    """The norm's codes as an operand of mx_gemm, and of the experts' grouped gate_up product with the router's rows: the
    bits of the norm and the quantizer called one by one."""
    m, rng = _m(), np.random.default_rng(10)
    T, H, N, EX, k = 96, 256, 128, 8, 2
    x, r = (to_dev_bf16(R.bf16(rng, (T, H))) for _ in range(2))
    w = to_dev_bf16(F.bf16_rne(1 + 0.1 * rng.standard_normal(H)))
    fm, lay = m.Format[fmt], m.Layout[layout]
    gs = m.GScale.PER_ROW if fmt == "NVFP4" else m.GScale.NONE
    say(f"norm to product {fmt} {layout}")
    n = m.mx_rmsnorm(x, w, EPS, residual=r, fmt=fm, layout=lay)
    y = m.mx_rmsnorm(x, w, EPS, residual=r).y
    q = (m.nvfp4_quantize(y, layout=lay) if fmt == "NVFP4" else m.mx_quantize(y, layout=lay)) + (None,)
    fused, apart = (m.Operand(fm, c, s, g, gs=gs, layout=lay) for c, s, g in ((n.codes, n.scales, n.gscales), q[:3]))
    wb = to_dev_bf16(R.bf16(rng, (N, H), 0.02))
    if fmt == "NVFP4":
        b = m.Operand(fm, *m.nvfp4_quantize(wb, gs=m.GScale.PER_TENSOR), gs=m.GScale.PER_TENSOR)
    else:
        b = m.Operand(fm, *m.mx_quantize(wb))
    assert torch.equal(m.mx_gemm(fused, b, T, N, H), m.mx_gemm(apart, b, T, N, H))
    if fmt != "NVFP4":
        return
    gate_up = D.Weight(rng, N, H, groups=EX).operand(m, torch)
    rt = m.mx_moe_route(torch.from_numpy(rng.standard_normal((T, EX)).astype(np.float32)).cuda(), k)
    kw = dict(group_row_offsets=rt.offsets, a_row_index=rt.row_token, a_rows=T)
    h = [m.mx_gemm_swiglu(a, gate_up, T * k, N // 2, H, **kw) for a in (fused, apart)]
    assert torch.equal(*h)
    out = m.mx_moe_combine(h[0], rt.row_of, rt.weights)
    ref, tol = R.combine_ref(_f64(h[0]), to_np(rt.row_of), to_np(rt.weights).astype(np.float64))
    assert (np.abs(_f64(out) - ref) <= tol).all()


def test_gradients_of_the_chain():
    """norm -> router and dispatched rows -> one product per expert (BF16 mx_gemm) -> combine, and back to the norm's input, its
    weight and the logits, against float64.  Seven BF16 roundings stand one behind the other, each at most 2^-8 of a value;
    the products and sums between mix values of both signs, so the norm of what they add stays below their sum: 7 2^-8
    of the result's norm, and as much again for the values that they are multiplied with."""
    m, rng = _m(), np.random.default_rng(9)
    T, H, N, EX, k = 96, 128, 128, 8, 2
    x, r, w = R.bf16(rng, (T, H)), R.bf16(rng, (T, H)), F.bf16_rne(1 + 0.1 * rng.standard_normal(H))
    W = F.bf16_rne(rng.standard_normal((EX, N, H)) * H ** -0.5)
    logits, dout = rng.standard_normal((T, EX)).astype(np.float32), R.bf16(rng, (T, N))
    xd, rd, wd, dd = (to_dev_bf16(a) for a in (x, r, w, dout))
    ld = torch.from_numpy(logits).cuda()
    B = lambda t, **kw: m.Operand(m.Format.BF16, t, block=m.Block.NONE, **kw)
    wt = to_dev_bf16(W)
    say("gradient chain")
    n = m.mx_rmsnorm(xd, wd, EPS, residual=rd, with_rstd=True)
    rt = m.mx_moe_route(ld, k)
    rows = m.mx_moe_dispatch(n.y, rt.row_of)
    y = m.mx_gemm(B(rows), B(wt.view(-1, H)), T * k, N, H, group_row_offsets=rt.offsets)
    out = m.mx_moe_combine(y, rt.row_of, rt.weights)
    dy, dw = m.mx_moe_combine_backward(dd, y, rt.row_of, rt.weights)
    dl = m.mx_moe_route_backward(dw, ld, rt.experts, rt.weights)
    drows = m.mx_gemm(B(dy), B(wt.transpose(1, 2).contiguous().view(-1, N)), T * k, H, N, group_row_offsets=rt.offsets)
    dn = m.mx_moe_combine(drows, rt.row_of)
    dx, dnw = m.mx_rmsnorm_backward(dn, n.h, wd, n.rstd)

    X = torch.tensor(R.f64(x) + R.f64(r), requires_grad=True)
    Wn = torch.tensor(R.f64(w), requires_grad=True)
    L = torch.tensor(logits.astype(np.float64), requires_grad=True)
    ids = rt.experts.cpu().long()
    yn = X / torch.sqrt((X * X).mean(1, keepdim=True) + EPS) * Wn
    p = torch.softmax(L.gather(1, ids), 1)
    We = torch.tensor(R.f64(W))
    ref = sum(p[:, j, None] * (We[ids[:, j]] @ yn[:, :, None])[..., 0] for j in range(k))
    ref.backward(torch.tensor(R.f64(dout)))
    off = lambda got, want: np.linalg.norm(got - want.numpy()) / np.linalg.norm(want.numpy())
    bound = 14 * R.EPS_BF16
    assert off(_f64(out), ref.detach()) <= bound
    assert off(_f64(dx), X.grad) <= bound and off(to_np(dnw), Wn.grad) <= bound and off(to_np(dl), L.grad) <= bound
