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
