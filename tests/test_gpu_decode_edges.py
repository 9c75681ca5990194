"""Calls of the decode step that stand at the edge of what the declarations allow."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests import decode_ref as R
from tests.test_gpu_attention import Problem
from tests.util import from_dev_bf16, requires_gpu, say, to_dev_bf16

pytestmark = [pytest.mark.gpu, requires_gpu]


def _m():
    import microscaling_quantization_block_amd as m
    return m


def _dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


@pytest.mark.parametrize("lens,split", [([900, 30], True), ([60, 30], False)])
@pytest.mark.parametrize("offs,none", [([0, 1, 4], 1), ([0, 1, 2 ** 31 - 1], 1), ([-2, 1, 3], 0)])
def test_offsets_outside_the_call(lens, split, offs, none):
    """A request whose offsets leave [0, tokens] has no rows, in the attention (split or not) and in the append; the
    other one is answered as ever."""
    m = _m()
    p = Problem(20, 64, 1, 2, 16, lens, [1, 2])
    need = m.nvfp4_attention_workspace(3, 2, 1, 64, 16, p.table.shape[1], 2, True)
    assert (need > 0) == split
    ws = torch.full((max(need, 1),), 0x7F, dtype=torch.uint8, device="cuda")     # not a row's place in it
    q, cache, table = to_dev_bf16(p.q), p.cache.device(m, torch), _dev(p.table)
    want, want_lse = p.run()
    out = torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 2), 6.0, device="cuda")
    say(f"offsets {offs} of 3 rows, lens {lens}")
    m.nvfp4_attention(q, cache, table, _dev(lens), q_offsets=_dev(offs), out=out, lse=lse, workspace=ws)
    gone = slice(1, 3) if none else slice(0, 1)
    here = slice(0, 1) if none else slice(1, 3)
    assert (out[gone] == 5.0).all() and (lse[gone] == 6.0).all()
    assert torch.equal(out[here], want[here]) and torch.equal(lse[here], want_lse[here])
    before = cache.k_codes.clone(), cache.v_gscales.clone()
    kv = torch.full((3, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    kd, vd = torch.full((2, 3, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda").unbind(0)
    m.nvfp4_cache_append(kv, kv, cache, table, _dev(lens), q_offsets=_dev(offs), k_dq=kd, v_dq=vd)
    assert (kd[gone] == 7.0).all() and (vd[gone] == 7.0).all() and (kd[here] == 2.0).all() and (vd[here] == 2.0).all()
    changed = (cache.k_codes != before[0]).any(-1)
    assert changed.sum() == (1 if none else 2)
    assert not torch.equal(cache.v_gscales, before[1])


# few columns unsplit, split; many columns unsplit, split; many columns with one KV head per query head
SHAPES = [([40, 33], [3, 2], 4), ([3000, 40], [1, 1], 4), ([300, 90], [1, 70], 4), ([3000], [150], 4), ([700], [600], 1)]


def _shape(seed, lens, news, grp, d=128, **kw):
    p = Problem(seed, d, 1, grp, 16, lens, news, **kw)
    return p, p.cache.device(_m(), torch)


def _call(p, cache, q=None):
    say(f"lens {p.lens} new {p.news} window {p.window} grp {p.grp} d {p.d}")
    return _m().nvfp4_attention(to_dev_bf16(p.q) if q is None else q, cache, _dev(p.table), _dev(p.lens),
                                q_offsets=_dev(p.offs), scale=p.scale, window=p.window, with_lse=True)


def _place(p, t, b=0):
    """Page and slot of token t of request b."""
    return int(p.table[b, t // p.page]), t % p.page


def _sees(p, t, b=0):
    """Which rows of the call have token t of request b in reach."""
    rows = torch.zeros(p.total, dtype=torch.bool, device="cuda")
    for i in range(p.news[b]):
        pos = p.lens[b] - p.news[b] + i
        rows[p.offs[b] + i] = t <= pos and (not p.window or t > pos - p.window)
    return rows


def _check_others(p, sees, out, lse, want, want_lse):
    """The rows that do not see the spoilt token are within their bounds (the others replaced by the clean call's)."""
    pick = sees[:, None]
    p.check(torch.where(pick[..., None], want, out), torch.where(pick, want_lse, lse))


@pytest.mark.parametrize("lens,news,grp", SHAPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_spoilt_query_row_is_nan(lens, news, grp, bad):
    """An infinity or a NaN in a row and head makes its output and its log sum NaN, however the context is cut."""
    p, cache = _shape(21, lens, news, grp)
    q = to_dev_bf16(p.q)
    row, head = 0, grp - 1
    q[row, head, 7] = bad
    # every key has the same sign there: infinite logits of one sign, no NaN among them
    p.cache.t["k_codes"][..., 3] = (p.cache.t["k_codes"][..., 3] & 0x0F) | 0x20
    cache = p.cache.device(_m(), torch)
    out, lse = _call(p, cache, q)
    assert out[row, head].isnan().all() and lse[row, head].isnan()
    out[row, head], lse[row, head] = 0.0, 0.0
    assert out.isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("lens,news,grp", SHAPES)
def test_a_spoilt_key_is_nan_where_it_is_seen(lens, news, grp):
    """A key whose second scale is NaN: the rows that reach it are NaN, log sum too; the others stand."""
    p, cache = _shape(22, lens, news, grp)
    want, want_lse = _call(p, cache)
    for t in {5, lens[0] - (news[0] + 1) // 2}:
        page, slot = _place(p, t)
        keep = cache.k_gscales[page, 0, slot].clone()
        cache.k_gscales[page, 0, slot] = float("nan")
        out, lse = _call(p, cache)
        cache.k_gscales[page, 0, slot] = keep
        sees = _sees(p, t)
        assert sees.any() and out[sees].isnan().all() and lse[sees].isnan().all(), t
        _check_others(p, sees, out, lse, want, want_lse)


@pytest.mark.parametrize("lens,news,grp", SHAPES)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("which", ["k", "v"])
def test_an_infinite_row_is_stored_as_nan(lens, news, grp, bad, which):
    """A K or V row with an infinity or a NaN has a NaN second scale: its values are NaN, and so is what sees it."""
    m = _m()
    p, cache = _shape(23, lens, news, grp)
    t = lens[0] - news[0]                                     # the first new token: every new row sees it
    page, slot = _place(p, t)
    rows = {n: torch.ones((1, 1, 128), dtype=torch.bfloat16, device="cuda") for n in "kv"}
    rows[which][0, 0, 77] = bad
    say(f"appended {which} {bad}")
    kd, vd = m.nvfp4_cache_append(rows["k"], rows["v"], cache, _dev(p.table[:1]), _dev([t + 1]), with_dq=True)
    S = cache.k_gscales if which == "k" else cache.v_gscales
    assert S[page, 0, slot].isnan() and (kd if which == "k" else vd).isnan().all()
    assert (vd if which == "k" else kd).isfinite().all()
    out, lse = _call(p, cache)
    rows = slice(p.offs[0], p.offs[1])
    assert out[rows].isnan().all() and not out[p.offs[1]:].isnan().any()
    assert lse[rows].isnan().all() if which == "k" else lse.isfinite().all()


# several rows of a request, which see different tokens: drafted tokens and prompt chunks, whole and split, windows
# that have passed a token for some rows only
UNEVEN = [([40, 33], [3, 2], 4, 0, 128), ([40], [16], 1, 0, 64), ([3000], [7], 4, 0, 128), ([90], [9], 1, 20, 256),
          ([70, 33], [30, 2], 2, 17, 128), ([300, 90], [100, 70], 4, 0, 128), ([3000], [150], 4, 0, 128),
          ([700], [600], 1, 0, 64), ([700], [300], 4, 100, 128), ([2000], [400], 2, 333, 64), ([400], [150], 2, 90, 256),
          ([3000], [300], 1, 900, 128), ([1500], [700], 1, 800, 256)]


def _spoilt_tokens(p):
    """Tokens that some rows of request 0 see and others do not: new ones, and ones that the window passes."""
    n, new = p.lens[0], p.news[0]
    for t in sorted({n - 1, n - (new + 1) // 2, n - new + 1} | ({n - new - p.window + 1 + new // 2} if p.window else set())):
        sees = _sees(p, t)
        yield t, sees
        assert sees.any() and not sees[p.offs[0]:p.offs[1]].all()


@pytest.mark.parametrize("lens,news,grp,window,d", UNEVEN)
@pytest.mark.parametrize("kind", ["second scale", "block scale", "infinite"])
def test_a_spoilt_value_is_kept_from_the_rows_that_do_not_see_it(kind, lens, news, grp, window, d):
    """A NaN in a token's V row (by its second scale, or by the scale of a block) reaches the rows that see the token
    and no others."""
    p, cache = _shape(24, lens, news, grp, d=d, window=window)
    want, want_lse = _call(p, cache)
    p.check(want, want_lse)
    for t, sees in _spoilt_tokens(p):
        page, slot = _place(p, t)
        at = cache.v_scales[page, 0, d // 16 - 1] if kind == "block scale" else cache.v_gscales[page, 0]
        keep = at[slot].clone()
        at[slot] = {"second scale": float("nan"), "infinite": float("inf"), "block scale": 0x7F}[kind]
        out, lse = _call(p, cache)
        at[slot] = keep
        spoilt = ~out[sees].isfinite()
        assert spoilt[..., -16:].all() if kind == "block scale" else spoilt.all(), t
        _check_others(p, sees, out, want_lse, want, want_lse)
        p.check(torch.where(sees[:, None, None], want, out), lse)      # log sums do not depend on V


@pytest.mark.parametrize("lens,news,grp,window,d", UNEVEN)
@pytest.mark.parametrize("power", [20, 60, 110])
def test_a_large_value_costs_the_rows_that_do_not_see_it_nothing(power, lens, news, grp, window, d):
    """One V row 2^power times the others: the bounds go by what a row sees."""
    p, cache = _shape(25, lens, news, grp, d=d, window=window)
    for t, sees in _spoilt_tokens(p):
        page, slot = _place(p, t)
        cache.v_gscales[page, 0, slot] *= 2.0 ** power
        p.v[0][:, t] *= 2.0 ** power
        out, lse = _call(p, cache)
        cache.v_gscales[page, 0, slot] *= 2.0 ** -power
        p.check(out, lse)
        p.v[0][:, t] *= 2.0 ** -power


def test_one_row_of_any_stride():
    """A size of one has a stride that means nothing: one row of x, of y, of q, one head."""
    m, rng = _m(), np.random.default_rng(26)
    n, k = 48, 64
    w = R.Weight(rng, n, k)
    x = to_dev_bf16(R.bf16(rng, (1, k)))
    odd = torch.empty_strided((1, k), (3, 1), dtype=torch.bfloat16, device="cuda").copy_(x)
    out = torch.empty_strided((1, n), (1, 1), dtype=torch.bfloat16, device="cuda")
    say("one row")
    want = m.nvfp4_gemv(x, w.operand(m, torch), 1, n, k)
    m.nvfp4_gemv(odd, w.operand(m, torch), 1, n, k, out=out)
    assert torch.equal(out, want)
    p = Problem(27, 64, 1, 1, 16, [40], [1])
    cache = p.cache.device(m, torch)
    q = to_dev_bf16(p.q)
    odd = torch.empty_strided((1, 1, 64), (3, 5, 1), dtype=torch.bfloat16, device="cuda").copy_(q)
    out = torch.empty_strided((1, 1, 64), (7, 9, 1), dtype=torch.bfloat16, device="cuda")
    args = cache, _dev(p.table), _dev(p.lens)
    want = m.nvfp4_attention(q, *args)
    m.nvfp4_attention(odd, *args, out=out)
    assert torch.equal(out, want)
    m.nvfp4_cache_append(odd, odd, *args)


@pytest.mark.parametrize("d,news,window", [(64, [90, 2], 0), (128, [90, 40], 0), (128, [200], 60), (256, [70, 1], 0),
                                           (128, [2, 3], 0)])
def test_holes_among_seen_tokens(d, news, window):
    """Pages missing in the middle of contexts that many columns see, with a NaN and a large V row around them."""
    lens = [250, 77][:len(news)]
    table = np.full((len(news), 16), -1, np.int32)
    table[0] = [0, 1, -1, 3, 4, 99, 5, 6, -7, 7, 8, -1, 9, 10, 11, 12]
    if len(news) > 1:
        table[1, :5] = [13, -1, 14, 15, 16]
    p = Problem(28, d, 1, 2, 16, lens, news, window=window, table=table, pages=17)
    cache = p.cache.device(_m(), torch)
    want, want_lse = _call(p, cache)
    p.check(want, want_lse)
    t = lens[0] - 1
    page, slot = _place(p, t)
    sees = _sees(p, t)
    for bad in (float("nan"), 2.0 ** 80):
        cache.v_gscales[page, 0, slot] = bad
        out, lse = _call(p, cache)
        assert out[sees].isnan().any() == (bad != bad)
        _check_others(p, sees, out, lse, want, want_lse)


@pytest.mark.parametrize("lens,news,grp", SHAPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_beyond_binary32_are_nan(lens, news, grp, sign):
    """q . k of 2^140: no finite logit, so no finite answer (and not that of an empty context)."""
    p, _ = _shape(29, lens, news, grp, k_scale=2.0 ** 70)
    p.scale = sign
    p.cache.t["k_codes"][...] &= 0x77                         # all keys positive
    q = to_dev_bf16(p.q)
    q[0, 0] = 2.0 ** 70
    out, lse = _call(p, p.cache.device(_m(), torch), q)
    assert out[0, 0].isnan().all() and lse[0, 0].isnan()
