"""Attention over the NVFP4 cache against float64 (bounds: tests/decode_ref.py).  Unused cache places hold 0xFF bytes
(NaN scales) unless a test says otherwise."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests import decode_ref as R
from tests.util import from_dev_bf16, requires_gpu, say, to_dev_bf16

pytestmark = [pytest.mark.gpu, requires_gpu]


def _m():
    import microscaling_quantization_block_amd as m
    return m


def _dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


class Problem:
    """Requests with a cache on the host; `kv` maps (request) -> k, v values [H, L, D] in float64."""

    def __init__(self, seed, d, heads, grp, page, lens, news, window=0, scale=None, k_scale=1.0, v_scale=None,
                 q_scale=1.0, pad=(0, 0), width_extra=0, table=None, pages=None):
        rng = np.random.default_rng(seed)
        self.d, self.heads, self.grp, self.page, self.lens, self.news = d, heads, grp, page, lens, news
        self.window, self.scale = window, d ** -0.5 if scale is None else scale
        if table is None:
            table, pages = R.tables(rng, lens, page, width_extra=width_extra)
        self.table = table
        self.cache = R.Cache(pages, heads, page, d)
        self.k, self.v, self.seen = [], [], []
        for b, n in enumerate(lens):
            kb = R.bf16(rng, (n, heads, d), k_scale)
            vb = R.bf16(rng, (n, heads, d))
            if v_scale is not None:                       # a magnitude per token
                vb = F.bf16_rne(F.bf16_bits_to_f64(vb) * v_scale(n)[:, None, None])
            kd, vd = np.zeros((2, heads, n, d))
            seen = np.zeros(n, bool)
            for t in range(n):
                p = table[b, t // page] if t // page < table.shape[1] else -1
                seen[t] = 0 <= p < pages
                kd[:, t] = self.cache.put("k", p if seen[t] else None, t % page, kb[t])
                vd[:, t] = self.cache.put("v", p if seen[t] else None, t % page, vb[t])
            self.k.append(kd)
            self.v.append(vd)
            self.seen.append(seen)
        self.offs = pad[0] + np.concatenate([[0], np.cumsum(news)])
        self.total = pad[0] + sum(news) + pad[1]
        self.q = R.bf16(rng, (self.total, heads * grp, d), q_scale)

    def run(self, ragged=True, q=None, **kw):
        m = _m()
        say(f"attention d {self.d} heads {self.heads}x{self.grp} page {self.page} lens {self.lens[:6]} "
            f"new {self.news[:6]} window {self.window} ragged {ragged}")
        return m.nvfp4_attention(to_dev_bf16(self.q) if q is None else q, self.cache.device(m, torch),
                                 _dev(self.table), _dev(self.lens),
                                 q_offsets=_dev(self.offs) if ragged else None, scale=self.scale, window=self.window,
                                 with_lse=True, **kw)

    def check(self, out, lse):
        got = F.bf16_bits_to_f64(from_dev_bf16(out))
        lse = lse.cpu().numpy().astype(np.float64)
        qv = F.bf16_bits_to_f64(self.q)
        for b, (n, new) in enumerate(zip(self.lens, self.news)):
            pos = n - new + np.arange(new)
            rows = slice(self.offs[b], self.offs[b + 1])
            for h in range(self.heads * self.grp):
                kv = h // self.grp
                o, s, to, ts = R.attention_ref(qv[rows, h], self.k[b][kv], self.v[b][kv], pos, self.scale, self.window,
                                               self.seen[b])
                e = np.abs(got[rows, h] - o)
                assert (e <= to).all(), (b, h, np.nanmax(e / np.maximum(to, 1e-300)), np.isnan(got[rows, h]).sum())
                with np.errstate(invalid="ignore"):
                    same = (lse[rows, h] == s) | (np.abs(lse[rows, h] - s) <= ts)
                assert same.all(), (b, h, lse[rows, h], s)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,grp", [(1, 1), (2, 4), (1, 5), (2, 16), (1, 24), (1, 40)])
@pytest.mark.parametrize("page", [16, 64])
def test_single_tokens(d, heads, grp, page):
    """One query per request; lengths of one token, of part of a page or a tile, of several."""
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 100, 257]
    p = Problem(d + grp, d, heads, grp, page, lens, [1] * len(lens))
    p.check(*p.run(ragged=False))


@pytest.mark.parametrize("d,grp", [(64, 4), (128, 4), (256, 2), (128, 1), (64, 3), (128, 16)])
@pytest.mark.parametrize("news", [[1, 5, 3, 1], [40, 1, 17, 64], [0, 70, 0, 2]])
def test_ragged_queries(d, grp, news):
    """Drafted tokens and prompt chunks: causal inside the new tokens, an empty request among them."""
    lens = [n + c for n, c in zip(news, [0, 33, 128, 7])]
    p = Problem(sum(news) + d, d, 2, grp, 16, lens, news)
    p.check(*p.run())


@pytest.mark.parametrize("window", [1, 16, 33, 100])
@pytest.mark.parametrize("d,news", [(64, [1, 1, 1]), (128, [1, 5, 2]), (128, [60, 1, 33])])
def test_window(d, news, window):
    lens = [max(n, c) for n, c in zip(news, [300, 90, 33])]
    p = Problem(window + d, d, 2, 2, 16, lens, news, window=window)
    p.check(*p.run())


@pytest.mark.parametrize("lens,new", [([1500, 700, 1], 1), ([5000], 1), ([3001, 64], 9), ([2600], 150)])
@pytest.mark.parametrize("d", [64, 128])
def test_split_contexts(d, lens, new):
    """Few requests of long contexts: several workgroups share one, a second launch joins them."""
    m = _m()
    news = [min(new, n) for n in lens]
    p = Problem(d + new, d, 1, 4, 32, lens, news)
    need = m.nvfp4_attention_workspace(sum(news), 4, 1, d, 32, p.table.shape[1], len(lens), new > 1)
    assert need > 0
    p.check(*p.run(ragged=new > 1))


def test_rows_that_see_nothing():
    """No context, more rows than tokens, no pages: zeros and -inf; rows of no request are left alone."""
    table = np.array([[-1, -1], [0, -1], [1, 2], [-1, 3]], np.int32)
    p = Problem(1, 128, 1, 4, 16, [0, 3, 20, 20], [2, 5, 1, 3], table=table, pages=4, pad=(1, 2))
    m = _m()
    out = torch.full((p.total, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.total, 4), 6.0, device="cuda")
    p.run(out=out, lse=lse)
    p.check(out, lse)
    assert (out[0] == 5.0).all() and (out[-2:] == 5.0).all() and (lse[0] == 6.0).all() and (lse[-2:] == 6.0).all()
    assert (out[1:3] == 0).all() and torch.isinf(lse[1:3]).all()


def test_rows_of_no_request_with_splits():
    p = Problem(2, 64, 1, 2, 16, [900, 30], [1, 2], pad=(1, 3))
    out = torch.full((p.total, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.total, 2), 6.0, device="cuda")
    p.run(out=out, lse=lse)
    p.check(out, lse)
    assert (out[0] == 5.0).all() and (out[-3:] == 5.0).all() and (lse[0] == 6.0).all() and (lse[-3:] == 6.0).all()


def test_holes_and_wide_tables():
    """Pages that are missing in the middle, entries outside the cache, a table wider than any request."""
    table = np.array([[0, -1, 2, 77, 1, -5], [3, 4, 5, -1, -1, -1]], np.int32)
    p = Problem(3, 128, 2, 2, 16, [75, 40], [3, 1], table=table, pages=6)
    p.check(*p.run())
    p = Problem(4, 64, 1, 4, 16, [75, 130, 9], [1, 1, 1], width_extra=200)
    p.check(*p.run(ragged=False))


def test_longer_than_the_table():
    """A length beyond the table's row: what lies beyond has no page."""
    p = Problem(5, 64, 1, 2, 16, [100], [1], table=np.array([[1, 0, 2]], np.int32), pages=3)
    p.check(*p.run(ragged=False))


@pytest.mark.parametrize("spread", [2.0 ** 12, 2.0 ** 25])
def test_second_scales_of_v(spread):
    """V rows of very different magnitude, growing and shrinking along the context."""
    up = lambda n: spread ** (np.arange(n) / max(n - 1, 1) - 0.5)
    for f in (up, lambda n: up(n)[::-1]):
        p = Problem(6, 128, 1, 4, 16, [200, 65], [1, 2], v_scale=f)
        p.check(*p.run())


@pytest.mark.parametrize("q_scale,k_scale", [(30.0, 30.0), (2.0 ** -60, 1.0), (2.0 ** 60, 2.0 ** -60), (0.0, 1.0)])
def test_logit_range(q_scale, k_scale):
    """One key takes all the weight; tiny and compensating magnitudes; zero queries (a plain mean)."""
    p = Problem(7, 128, 1, 4, 16, [90, 33], [1, 4], q_scale=q_scale, k_scale=k_scale)
    p.check(*p.run())


def test_scale_argument():
    p = Problem(8, 64, 2, 2, 16, [50], [3], scale=-0.3)
    p.check(*p.run())


def test_strided_rows():
    """q as a slice of a fused projection, out as a slice of a wider buffer."""
    p = Problem(9, 64, 2, 2, 16, [50, 20], [2, 3])
    hq = 4
    fused = torch.zeros((p.total, 8, 64), dtype=torch.bfloat16, device="cuda")
    fused[:, :hq] = to_dev_bf16(p.q)
    wide = torch.full((p.total, hq, 3, 64), 4.0, dtype=torch.bfloat16, device="cuda")
    out, lse = p.run(q=fused[:, :hq], out=wide[:, :, 1])
    p.check(out, lse)
    assert (wide[:, :, 0] == 4.0).all() and (wide[:, :, 2] == 4.0).all()


def test_equal_calls_give_equal_bits_with_a_used_workspace():
    m = _m()
    p = Problem(10, 128, 1, 4, 32, [2000, 300], [1, 1])
    ws = torch.full((m.nvfp4_attention_workspace(2, 4, 1, 128, 32, p.table.shape[1], 2, False),), 255,
                    dtype=torch.uint8, device="cuda")
    a, la = p.run(ragged=False, workspace=ws)
    b, lb = p.run(ragged=False, workspace=ws)
    p.check(a, la)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_empty_calls():
    m = _m()
    cache = m.NVFP4Cache.empty(2, 1, 16, 64)
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = m.nvfp4_attention(q, cache, torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                            torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 2, 64)


@pytest.mark.parametrize("news", [[1, 1], [3, 70]])
def test_windows_wider_than_any_context(news):
    p = Problem(11, 64, 1, 2, 16, [300, 90], news)
    a, la = p.run()
    for p.window in (1 << 31, (1 << 32) + 3, (1 << 63) - 1):
        b, lb = p.run()
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("lens,news", [([40, 33], [3, 2]), ([300, 90], [1, 70]), ([3000, 40], [1, 1])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_spoilt_query_row_stays_by_itself(lens, news, bad):
    """An infinity or a NaN in one row and head leaves every other row and head as it was."""
    p = Problem(12, 128, 1, 4, 16, lens, news)
    a, la = p.run()
    q = to_dev_bf16(p.q)
    row, head = p.total - 1, 2
    q[row, head, 7] = bad
    b, lb = p.run(q=q)
    keep = torch.ones(p.total, 4, dtype=torch.bool, device="cuda")
    keep[row, head] = False
    assert torch.equal(a[keep], b[keep]) and torch.equal(la[keep], lb[keep])


@pytest.mark.parametrize("new", [1, 90])
def test_shared_pages_and_a_page_named_twice(new):
    """Two requests over the same pages answer alike; a table that names a page twice reads it twice."""
    p = Problem(13, 64, 2, 2, 16, [128], [new])
    table = np.concatenate([p.table, p.table])
    q = to_dev_bf16(np.concatenate([p.q, p.q]))
    m = _m()
    cache = p.cache.device(m, torch)
    say(f"shared pages {new}")
    out = m.nvfp4_attention(q, cache, _dev(table), _dev([128, 128]), q_offsets=_dev([0, new, 2 * new]))
    assert torch.equal(out[:new], out[new:])
    p.check(out[:new], p.run()[1])
    p.table = np.concatenate([p.table[:, :4], p.table[:, :4]], 1)
    p.k = [np.concatenate([x[:, :64], x[:, :64]], 1) for x in p.k]
    p.v = [np.concatenate([x[:, :64], x[:, :64]], 1) for x in p.v]
    p.check(*p.run())


@pytest.mark.parametrize("new", [1, 40, 300])
def test_pages_far_apart(new):
    """Pages a gibibyte apart: byte offsets beyond 32 bits, in the append too."""
    m, rng = _m(), np.random.default_rng(14)
    h, page, d, pages, far = 2, 16, 128, 6, 1 << 30
    n = page * pages * 4 if new > 90 else page * pages
    if n > page * pages:                                       # more tokens: the same pages with more slots
        page *= 4
    big = [torch.empty((pages - 1) * far + h * page * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    codes = [b.as_strided((pages, h, page, d // 2), (far, page * d // 2, d // 2, 1)) for b in big]
    plain = m.NVFP4Cache.empty(pages, h, page, d)
    cache = m.NVFP4Cache(codes[0], plain.k_scales, plain.k_gscales, codes[1], plain.v_scales, plain.v_gscales)
    table = _dev(rng.permutation(pages)[None])
    k, v = (to_dev_bf16(R.bf16(rng, (n, h, d))) for _ in "kv")
    q = to_dev_bf16(R.bf16(rng, (new, 4 * h, d)))
    say(f"pages far apart {new}")
    got = []
    for c in (cache, plain):
        m.nvfp4_cache_append(k, v, c, table, _dev([n]), q_offsets=_dev([0, n]))
        got.append(m.nvfp4_attention(q, c, table, _dev([n]), q_offsets=_dev([0, new])))
    assert torch.equal(cache.k_codes, plain.k_codes) and torch.equal(cache.v_codes, plain.v_codes)
    assert torch.equal(got[0], got[1]) and not got[1].isnan().any()


@pytest.mark.parametrize("news", [[1, 1], [3, 2], [150, 60]])
@pytest.mark.parametrize("d,window", [(64, 100), (128, 700), (256, 300)])
def test_window_much_shorter_than_the_context(d, window, news):
    p = Problem(15, d, 1, 2, 16, [3000, 900], news, window=window)
    p.check(*p.run())


def test_many_short_contexts():
    """More requests than the chip has compute units, none longer than 2048 tokens: not split."""
    lens = [700, 1, 33, 0] + [40] * 300
    p = Problem(16, 64, 1, 2, 16, lens, [1] * len(lens))
    assert _m().nvfp4_attention_workspace(len(lens), 2, 1, 64, 16, p.table.shape[1], len(lens), False) == 0
    p.check(*p.run(ragged=False))
