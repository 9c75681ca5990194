"""Paths of the decode step that a call takes by its sizes alone: each choice of the launchers at least once."""

import numpy as np
import pytest
import torch

from tests import decode_ref as R
from tests.test_gpu_attention import Problem
from tests.test_gpu_cache import _run as _append
from tests.test_gpu_gemv import _dense
from tests.util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def _workspace(p, ragged=True):
    import microscaling_quantization_block_amd as m
    return m.nvfp4_attention_workspace(p.total, p.heads * p.grp, p.heads, p.d, p.page, p.table.shape[1], len(p.lens),
                                       ragged)


@pytest.mark.parametrize("lens,new", [([1500, 700, 1], 1), ([3001, 64], 9), ([2600], 150)])
def test_split_contexts_of_wide_heads(lens, new):
    """head_dim 256 split and joined, both kernels."""
    p = Problem(30 + new, 256, 1, 4, 32, lens, [min(new, n) for n in lens])
    assert _workspace(p) > 0
    p.check(*p.run())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_join_of_many_rows(d):
    """More than 4096 (row, head) pairs of split contexts: a wave per row in the join."""
    p = Problem(31, d, 1, 8, 64, [2800, 40], [560, 1])
    assert _workspace(p) > 0 and p.total * 8 > 4096
    p.check(*p.run())


@pytest.mark.parametrize("count,grp,d", [(70, 4, 64), (130, 2, 128)])
def test_many_requests_in_a_wide_table(count, grp, d):
    """More requests than a wave has lanes, split: the units of the later ones follow those of the earlier."""
    rng = np.random.default_rng(count)
    lens = [int(n) for n in rng.integers(1, 90, count)]
    lens[3], lens[count - 2], lens[66] = 700, 900, 0
    news = [1 + int(n) for n in rng.integers(0, 3, count)]
    p = Problem(32, d, 1, grp, 16, lens, news, width_extra=100)
    assert _workspace(p) > 0
    p.check(*p.run())
    p = Problem(33, d, 1, grp, 16, lens, [1] * count, width_extra=100)
    assert _workspace(p, False) > 0
    p.check(*p.run(ragged=False))


def test_more_chunks_than_lanes():
    """A context of more than 64 chunks."""
    p = Problem(34, 64, 1, 2, 64, [18000], [1])
    assert _workspace(p, False) > 0
    p.check(*p.run(ragged=False))


@pytest.mark.parametrize("page", [256, 1024])
@pytest.mark.parametrize("news", [[1, 1], [3, 90]])
def test_large_pages(page, news):
    p = Problem(35, 128, 2, 2, page, [1300, 300], news)
    p.check(*p.run())


@pytest.mark.parametrize("page", [256, 1024])
@pytest.mark.parametrize("d", [64, 256])
def test_append_to_large_pages(d, page):
    rng = np.random.default_rng(page)
    lens, news = [1100, 20], [40, 3]
    _append(rng, 2, d, page, lens, news, R.bf16(rng, (43, 2, d)), R.bf16(rng, (43, 2, d)), True)


LAYOUTS = [("row", "linear"), ("row", "mfma"), ("tile", "linear")]


@pytest.mark.parametrize("m_rows,k", [(5, 1088), (16, 1536), (3, 2048), (16, 2048)])
@pytest.mark.parametrize("block,layout", LAYOUTS)
@pytest.mark.parametrize("op", ["gemv", "swiglu"])
def test_streamed_rows_between_one_and_two_thousand(op, block, layout, m_rows, k):
    _dense(op, m_rows, 96, k, block, layout, m_rows + k)


@pytest.mark.parametrize("k", [768, 1088, 4096, 14336])
@pytest.mark.parametrize("block,layout", LAYOUTS)
@pytest.mark.parametrize("op", ["gemv", "swiglu"])
def test_two_rows_of_longer_weights(op, block, layout, k):
    _dense(op, 2, 96, k, block, layout, k)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,news,grp", [([257, 100, 33], [1, 1, 1], 4), ([300, 64], [3, 2], 2), ([2900], [1], 8)])
def test_few_columns_round_once(d, lens, news, grp):
    """The kernel for few columns rounds the weights to FP16 and nothing else: the values c s_b are FP16 numbers, and
    the second scale goes to the weight before it is rounded.  So one rounding of 2^-11 where decode_ref has three."""
    from oracle import formats as F
    from tests.util import from_dev_bf16
    p = Problem(36, d, 1, grp, 32, lens, news)
    out, lse = p.run()
    p.check(out, lse)
    got, qv = F.bf16_bits_to_f64(from_dev_bf16(out)), F.bf16_bits_to_f64(p.q)
    for b, (n, new) in enumerate(zip(lens, news)):
        rows, pos = slice(p.offs[b], p.offs[b + 1]), n - new + np.arange(new)
        for h in range(grp):
            o, _, tol, _ = R.attention_ref(qv[rows, h], p.k[b][0], p.v[b][0], pos, p.scale, 0)
            mass = R.attention_ref(qv[rows, h], p.k[b][0], np.abs(p.v[b][0]), pos, p.scale, 0)[0]
            tight = tol - (1 + R.EPS_BF16) * 2 * R.EPS_FP16 * mass
            assert (tight > 0).all() and (np.abs(got[rows, h] - o) <= tight).all(), (b, h)
