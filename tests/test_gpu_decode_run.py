"""The decode operators together: the step of a small 4-bit sampler, stage by stage against float64 on the stage's own
input; the step captured into a graph; calls on two streams at once."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests import decode_ref as R
from tests.util import from_dev_bf16, requires_gpu, say, to_dev_bf16

pytestmark = [pytest.mark.gpu, requires_gpu]

HID, HQ, HKV, D, INTER, PAGE = 256, 4, 2, 64, 192, 16


def _m():
    import microscaling_quantization_block_amd as m
    return m


def _f64(t):
    return F.bf16_bits_to_f64(from_dev_bf16(t))


class Sampler:
    """One layer: projections, cache, attention, gated MLP; residuals in torch."""

    def __init__(self, seed, lens, pages=40, width=8):
        rng = np.random.default_rng(seed)
        m = _m()
        self.w = dict(qkv=R.Weight(rng, (HQ + 2 * HKV) * D, HID), o=R.Weight(rng, HID, HQ * D, block="tile"),
                      gate_up=R.Weight(rng, 2 * INTER, HID, layout="mfma"), down=R.Weight(rng, HID, INTER))
        self.op = {k: w.operand(m, torch) for k, w in self.w.items()}
        self.b = len(lens)
        table = rng.permutation(pages)[:self.b * width].reshape(self.b, width).astype(np.int32)
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cache = m.NVFP4Cache.empty(pages, HKV, PAGE, D)
        for n in ("k_codes", "k_scales", "k_gscales", "v_codes", "v_scales", "v_gscales"):
            t = getattr(self.cache, n)
            t.view(torch.uint8).fill_(0xFF)               # stale pages
        prompt = max(lens) - 1
        n = [x - 1 for x in lens]                         # the prompts: all but the first decoded token
        offs = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device="cuda")
        kv = [to_dev_bf16(R.bf16(rng, (sum(n), HKV, D))) for _ in "kv"]
        m.nvfp4_cache_append(*kv, self.cache, self.table, self.lens - 1, q_offsets=offs)
        self.x = to_dev_bf16(R.bf16(rng, (self.b, HID)))
        assert prompt < width * PAGE

    def step(self, x):
        """The next hidden state; also every stage's input and output."""
        m, b = _m(), self.b
        qkv = m.nvfp4_gemv(x, self.op["qkv"], b, (HQ + 2 * HKV) * D, HID).view(b, -1, D)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        m.nvfp4_cache_append(k, v, self.cache, self.table, self.lens)
        att = m.nvfp4_attention(q, self.cache, self.table, self.lens)
        o = m.nvfp4_gemv(att.view(b, -1), self.op["o"], b, HID, HQ * D)
        r = x + o
        h = m.nvfp4_gemv_swiglu(r, self.op["gate_up"], b, INTER, HID)
        d = m.nvfp4_gemv(h, self.op["down"], b, HID, INTER)
        return r + d, dict(x=x, qkv=qkv.view(b, -1), att=att, o=o, r=r, h=h, d=d)


def _cached(s, name, b, ctx):
    """The first ctx rows of a request as the cache holds them, [HKV, ctx, D] float64."""
    from oracle import nvfp4 as ON
    c = s.cache
    codes = getattr(c, name + "_codes").cpu().numpy()
    scales = getattr(c, name + "_scales").cpu().numpy()
    gs = getattr(c, name + "_gscales").cpu().numpy()
    table = s.table.cpu().numpy()
    out = np.zeros((HKV, ctx, D))
    for t in range(ctx):
        p, slot = table[b, t // PAGE], t % PAGE
        sc = scales[p, :, slot] if name == "k" else scales[p, :, :, slot]
        out[:, t] = ON.dequantize_f64(codes[p, :, slot], sc, gs[p, :, slot], "1x16", "per_row")
    return out


def test_steps_stage_by_stage():
    s = Sampler(1, [1, 17, 40, 100])
    x = s.x
    for i in range(3):
        say(f"decode step {i}")
        nxt, st = s.step(x)
        for name, a, w in (("qkv", "x", "qkv"), ("o", "att", "o"), ("d", "h", "down")):
            ref, tol = R.gemv_ref(_f64(st[a].reshape(s.b, -1)), s.w[w].dq[0])
            assert (np.abs(_f64(st[name]) - ref) <= tol).all(), (i, name)
        gu = s.w["gate_up"].dq[0]
        ref, tol = R.swiglu_ref(_f64(st["r"]), gu[:INTER], gu[INTER:])
        assert (np.abs(_f64(st["h"]) - ref) <= tol).all(), i
        q, lens = _f64(st["qkv"]).reshape(s.b, -1, D)[:, :HQ], s.lens.cpu().numpy()
        att = _f64(st["att"])
        for b in range(s.b):
            k, v = _cached(s, "k", b, lens[b]), _cached(s, "v", b, lens[b])
            for h in range(HQ):
                o, _, tol, _ = R.attention_ref(q[b:b + 1, h], k[h // 2], v[h // 2], lens[b:b + 1] - 1, D ** -0.5, 0)
                assert (np.abs(att[b, h] - o[0]) <= tol[0]).all(), (i, b, h)
        x = nxt
        s.lens += 1


def test_captured_step():
    """A captured step advances the lengths itself; each replay equals the eager step, bit for bit, with eager work
    of the program between the replays.  Two graphs of the same sampler's shapes alternate."""
    lens = [5, 60, 31]
    eager, graphs = [Sampler(2, lens), Sampler(3, lens)], []
    say("capture")
    for seed in (2, 3):
        s = Sampler(seed, lens)
        buf = s.x.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.step(buf)                                    # warm up; writes the token that the first replay rewrites
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, _ = s.step(buf)
            buf.copy_(out)
            s.lens.add_(1)
        graphs.append((g, s, buf))
    xs = [e.x for e in eager]
    for i in range(5):
        for j in (0, 1):
            say(f"replay {i} of graph {j}")
            graphs[j][0].replay()
            xs[j], _ = eager[j].step(xs[j])
            eager[j].lens += 1
            torch.cuda.synchronize()
            assert torch.equal(graphs[j][2], xs[j]), (i, j)
            assert torch.equal(graphs[j][1].cache.v_scales, eager[j].cache.v_scales)


def test_two_streams_at_once():
    """Long contexts (split, with workspaces) on two streams in flight together equal the calls one by one."""
    m, rng = _m(), np.random.default_rng(4)
    pages, heads, d, page, b = 160, 2, 128, 32, 2
    cache = m.NVFP4Cache.empty(pages, heads, page, d)
    table = torch.from_numpy(rng.permutation(pages).reshape(b, -1).astype(np.int32)).cuda()
    lens = torch.tensor([2500, 1800], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, 2500, 4300], dtype=torch.int32, device="cuda")
    k, v = (to_dev_bf16(R.bf16(rng, (4300, heads, d))) for _ in "kv")
    m.nvfp4_cache_append(k, v, cache, table, lens, q_offsets=offs)
    qs = [to_dev_bf16(R.bf16(rng, (b, 8, d))) for _ in range(2)]
    want = [m.nvfp4_attention(q, cache, table, lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    say("two streams")
    for _ in range(5):
        got = [m.nvfp4_attention(q, cache, table, lens, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
