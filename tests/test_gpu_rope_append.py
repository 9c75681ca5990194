"""Rotary positions on the way into the cache: q bit for bit by the definition's steps, the cache's bytes those of
nvfp4_cache_append for the turned keys, everything else untouched."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests import decode_ref as D, layer_ref as R
from tests.util import from_dev_bf16, requires_gpu, say, to_dev_bf16

pytestmark = [pytest.mark.gpu, requires_gpu]

NAMES = ("k_codes", "k_scales", "k_gscales", "v_codes", "v_scales", "v_gscales")


def _m():
    import microscaling_quantization_block_amd as m
    return m


def _freq(rot, base=10000.0):
    return (base ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _run(rng, hq, h, d, page, lens, news, rot, interleaved, ragged=True, front=0, back=0, table=None, pages=None,
         factor=1.0, form="plain", q_bits=None, k_bits=None, freq=None):
    m = _m()
    if table is None:
        table, pages = D.tables(rng, lens, page, width_extra=1)
    total = front + sum(news) + back
    q = R.bf16(rng, (total, hq, d)) if q_bits is None else q_bits
    k = R.bf16(rng, (total, h, d)) if k_bits is None else k_bits
    v = R.bf16(rng, (total, h, d))
    offs = front + np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    pos, live = np.zeros(total, np.int64), np.zeros(total, bool)
    for b, (n, new) in enumerate(zip(lens, news)):
        pos[offs[b]:offs[b] + new] = n - new + np.arange(new)
        live[offs[b]:offs[b] + new] = True
    freq = _freq(rot) if freq is None else freq
    qt, kt = (R.turned_bits(x, pos, freq, interleaved, factor) for x in (q, k))
    host = D.Cache(pages, h, page, d, fill=0xA5)
    got, want = host.device(m, torch), host.device(m, torch)
    td, ld = _cuda(table), torch.tensor(lens, dtype=torch.int32, device="cuda")
    od = _cuda(offs) if ragged else None
    say(f"rope append q {hq} kv {h} d {d} rot {rot} page {page} lens {lens[:6]} new {news[:6]} interleaved {interleaved} {form}")
    wk, wv = (torch.full((total, h, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    m.nvfp4_cache_append(to_dev_bf16(kt), to_dev_bf16(v), want, td, ld, q_offsets=od, k_dq=wk, v_dq=wv)
    kd, vd = (torch.full((total, h, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kw = dict(q_offsets=od, interleaved=interleaved, factor=factor)
    if form == "fused":                                    # slices of one projection's output, q turned in place
        fused = torch.zeros((total, hq + 2 * h, d), dtype=torch.bfloat16, device="cuda")
        qd, kx, vx = fused[:, :hq], fused[:, hq:hq + h], fused[:, hq + h:]
        qd.copy_(to_dev_bf16(q))
        kx.copy_(to_dev_bf16(k))
        vx.copy_(to_dev_bf16(v))
        out, _, _ = m.nvfp4_rope_append(qd, kx, vx, got, td, ld, _cuda(freq), out=qd, k_dq=kd, v_dq=vd, **kw)
        assert torch.equal(kx, to_dev_bf16(k)) and torch.equal(vx, to_dev_bf16(v))
        rest = q
    else:
        out = torch.full((total, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
        rest = from_dev_bf16(out)
        args = (to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), got, td, ld, _cuda(freq))
        if form == "bare":
            assert m.nvfp4_rope_append(*args, out=out, **kw) is out
            kd, vd = wk, wv
        else:
            m.nvfp4_rope_append(*args, out=out, k_dq=kd, v_dq=vd, **kw)
    res = from_dev_bf16(out)
    same = (res == qt) | (np.isnan(R.f64(res)) & np.isnan(R.f64(qt)))
    assert same[live].all()
    assert np.array_equal(res[~live], rest[~live])
    byte = lambda t: t.contiguous().view(torch.uint8)
    # the sign of a NaN is not defined, and codes and BF16 values carry it: rows whose second scale is a NaN are NaN
    # whatever their codes hold (untouched places, 0xA5A5A5A5, are numbers)
    spoilt = torch.isnan(want.k_gscales)
    assert torch.equal(torch.isnan(got.k_gscales), spoilt)
    for n in NAMES:
        a, b = getattr(got, n), getattr(want, n)
        if n == "k_codes":
            a, b = a.masked_fill(spoilt[..., None], 0), b.masked_fill(spoilt[..., None], 0)
        assert torch.equal(byte(a), byte(b)), n
    assert torch.equal(kd.isnan(), wk.isnan()) and torch.equal(byte(kd.nan_to_num()), byte(wk.nan_to_num()))
    assert torch.equal(byte(vd), byte(wv))


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 96), (256, 256), (256, 32), (256, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,h", [(1, 1), (3, 1), (8, 8), (32, 8), (5, 5), (40, 4)])
def test_one_row_per_request(d, rot, interleaved, hq, h):
    rng = np.random.default_rng(d + rot + hq)
    lens = [1, 16, 17, 95, 7, 1000]
    _run(rng, hq, h, d, 16, lens, [1] * 6, rot, interleaved, ragged=False)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("form", ["plain", "bare", "fused"])
def test_prompts(d, page, interleaved, form):
    """Ragged rows with an empty request, rows before the first and behind the last one."""
    rng = np.random.default_rng(d)
    _run(rng, 6, 2, d, page, [37, 5, 18, 300], [37, 0, 1, 220], d, interleaved, front=2, back=3, factor=1.25, form=form)


def test_many_tokens():
    """More tokens than there are waves to share their heads: a wave holds all heads of a token."""
    _run(np.random.default_rng(2), 7, 3, 64, 32, [2500, 1800, 40], [2400, 1800, 1], 64, False)
    _run(np.random.default_rng(3), 2, 1, 128, 32, [4200], [4200], 64, True)


def test_rows_without_a_page():
    """Entries outside the cache, positions beyond the table, more rows than tokens: q is turned (at negative positions
    too), keys and values are not stored."""
    table = np.array([[0, -1, 2], [3, 99, 1], [4, 5, -2147483648]], np.int32)
    _run(np.random.default_rng(4), 4, 2, 64, 16, [40, 70, 2], [40, 30, 5], 64, False, table=table, pages=6)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Positions to 2^31 - 2, without a page there: the angles keep their digits.  Fast frequencies and one of 0."""
    lens = [2147483647, 1 << 30, 123456789, 1000003]
    freq = _freq(128)
    freq[3], freq[7], freq[9] = 0.0, 100.0, -0.75
    table = np.full((4, 2), -1, np.int32)
    _run(np.random.default_rng(5), 4, 2, 128, 16, lens, [1, 3, 2, 1], 128, interleaved, table=table, pages=1, freq=freq)


def test_magnitudes_and_spoilt_rows():
    """Zero rows, the smallest and largest values, an infinity and a NaN in one row: bits, and no other row's."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((8, 2, 128))
    x[0] = 0.0
    x[1] *= 2.0 ** -130
    x[2] *= 2.0 ** 120
    x[3] *= 2.0 ** -70
    bits = F.bf16_rne(x)
    bits[5, 0, 3], bits[6, 1, 70] = 0x7F80, 0x7FC0
    for inter in (False, True):
        _run(rng, 2, 2, 128, 16, [8], [8], 128, inter, q_bits=bits, k_bits=bits)


def test_strided_heads():
    """q [tokens, heads, d] stored head by head."""
    m, rng = _m(), np.random.default_rng(7)
    q = to_dev_bf16(R.bf16(rng, (3, 20, 64)))               # [heads, tokens, d]
    k, v = (to_dev_bf16(R.bf16(rng, (20, 1, 64))) for _ in "kv")
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    say("strided heads")
    f = _cuda(_freq(64))
    a, b = (m.NVFP4Cache.empty(2, 1, 16, 64) for _ in range(2))
    want = m.nvfp4_rope_append(q.transpose(0, 1).contiguous(), k, v, a, table, lens, f, q_offsets=offs)
    out = torch.empty_like(q)
    got = m.nvfp4_rope_append(q.transpose(0, 1), k, v, b, table, lens, f, q_offsets=offs, out=out.transpose(0, 1))
    assert torch.equal(got, want) and torch.equal(a.k_codes[table[0].long(), 0].flatten(0, 1)[:20], b.k_codes[table[0].long(), 0].flatten(0, 1)[:20])


def test_refusals():
    m = _m()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    cache = m.NVFP4Cache.empty(2, 1, 16, 64)
    t, n = torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    f = torch.ones(32, device="cuda")
    ok = (bf(3, 2, 64), bf(3, 1, 64), bf(3, 1, 64), cache, t, n, f)
    m.nvfp4_rope_append(*ok)
    for i, bad in ((0, bf(3, 2, 128)), (0, bf(2, 2, 64)), (1, bf(3, 2, 64)), (2, bf(4, 1, 64)), (0, bf(3, 64, 2).transpose(1, 2)),
                   (6, f[:33:2][:16]), (6, f.cpu())):
        with pytest.raises(ValueError):
            m.nvfp4_rope_append(*ok[:i], bad, *ok[i + 1:])
    for i, bad in ((0, ok[0].float()), (6, f.double()), (3, None), (1, None)):
        with pytest.raises(TypeError):
            m.nvfp4_rope_append(*ok[:i], bad, *ok[i + 1:])
    for bad in (f[:12], torch.ones(40, device="cuda"), f[:0]):
        with pytest.raises(m.MXQError):
            m.nvfp4_rope_append(*ok[:6], bad)
    with pytest.raises(m.MXQError):
        m.nvfp4_rope_append(*ok, factor=float("inf"))
    with pytest.raises(ValueError):
        m.nvfp4_rope_append(*ok, k_dq=bf(3, 2, 64)[:, :1])
