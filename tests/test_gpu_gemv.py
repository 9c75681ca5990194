"""Products of a few BF16 rows with NVFP4 weights against float64 (bounds: tests/decode_ref.py)."""

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


def _check(got, ref, tol, what):
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / np.maximum(tol, 1e-300))} bounds"


def _x(rng, m, k):
    return F.bf16_rne(rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1))))


def _dense(op, m_rows, n, k, block, layout, seed):
    m, rng = _m(), np.random.default_rng(seed)
    w = R.Weight(rng, 2 * n if op == "swiglu" else n, k, block, layout)
    x = _x(rng, m_rows, k)
    xv = F.bf16_bits_to_f64(x)
    say(f"{op} {m_rows} {n} {k} {block} {layout}")
    fn = m.nvfp4_gemv if op == "gemv" else m.nvfp4_gemv_swiglu
    y = fn(to_dev_bf16(x), w.operand(m, torch), m_rows, n, k)
    ref, tol = (R.gemv_ref(xv, w.dq[0]) if op == "gemv" else R.swiglu_ref(xv, w.dq[0][:n], w.dq[0][n:]))
    _check(F.bf16_bits_to_f64(from_dev_bf16(y)), ref, tol, (op, m_rows, n, k, block, layout))


@pytest.mark.parametrize("m_rows,n,k", [(1, 16, 16), (1, 1, 32), (2, 17, 48), (3, 40, 144), (5, 33, 272), (8, 64, 128),
                                        (16, 48, 1040), (17, 31, 2064), (33, 80, 496), (64, 100, 1024), (1, 50, 14336),
                                        (7, 4096, 256), (130, 20, 160)])
@pytest.mark.parametrize("op", ["gemv", "swiglu"])
def test_row_blocks(op, m_rows, n, k):
    _dense(op, m_rows, n, k, "row", "linear", m_rows * 1000 + n)


@pytest.mark.parametrize("m_rows,n,k", [(1, 16, 64), (4, 96, 320), (19, 32, 4096), (1, 2048, 768), (12, 256, 64)])
@pytest.mark.parametrize("block,layout", [("tile", "linear"), ("row", "mfma")])
@pytest.mark.parametrize("op", ["gemv", "swiglu"])
def test_tiles_and_mfma_scales(op, block, layout, m_rows, n, k):
    if layout == "mfma" and op == "gemv" and n % 32:
        n += 16
    _dense(op, m_rows, n, k, block, layout, m_rows * 1000 + n + 7)


def test_every_code_and_scale_exactly():
    """Unit rows of x pick single weights out: y is the dequantized weight, bit for bit, for every code under
    every finite E4M3 scale."""
    m = _m()
    k = 16
    scales = np.array([s for s in range(256) if s & 0x7F != 0x7F], np.uint8)
    n = scales.size
    codes = np.tile(np.array([(2 * j) | (2 * j + 1) << 4 for j in range(8)], np.uint8), (n, 1))
    dev = lambda a: torch.from_numpy(a).cuda()
    w = m.Operand(m.Format.NVFP4, dev(codes), dev(scales), torch.ones(1, device="cuda"), gs=m.GScale.GIVEN)
    say("gemv, every code and scale")
    y = m.nvfp4_gemv(torch.eye(16, dtype=torch.bfloat16, device="cuda"), w, 16, n, k)
    want = F.e2m1_value(np.arange(16))[:, None] * F.e4m3_value(scales)[None]
    assert np.array_equal(F.bf16_bits_to_f64(from_dev_bf16(y)), want)


@pytest.mark.parametrize("counts", [[1, 0, 3, 0], [0, 0, 0], [40, 1, 16, 17], [5]])
@pytest.mark.parametrize("op", ["gemv", "swiglu"])
@pytest.mark.parametrize("block,layout", [("row", "linear"), ("tile", "linear"), ("row", "mfma")])
def test_groups(op, block, layout, counts):
    m, rng = _m(), np.random.default_rng(sum(counts))
    n, k, e = 64, 192, len(counts)
    w = R.Weight(rng, 2 * n if op == "swiglu" else n, k, block, layout, groups=e)
    rows = sum(counts) + 2                                # two rows of no group at the end
    tokens = 6
    x = _x(rng, tokens, k)
    index = rng.integers(0, tokens, rows).astype(np.int32)
    if sum(counts) > 3:
        index[1], index[2] = -1, tokens                   # outside: a row of zeros
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    fn = m.nvfp4_gemv if op == "gemv" else m.nvfp4_gemv_swiglu
    say(f"groups {op} {block} {layout} {counts}")
    fn(to_dev_bf16(x), w.operand(m, torch), rows, n, k, out=out, group_row_offsets=torch.from_numpy(off).cuda(),
       x_row_index=torch.from_numpy(index).cuda())
    got = F.bf16_bits_to_f64(from_dev_bf16(out))
    xv = np.where(((index >= 0) & (index < tokens))[:, None], F.bf16_bits_to_f64(x)[index.clip(0, tokens - 1)], 0.0)
    for g in range(e):
        r = slice(off[g], off[g + 1])
        ref, tol = (R.gemv_ref(xv[r], w.dq[g]) if op == "gemv" else R.swiglu_ref(xv[r], w.dq[g][:n], w.dq[g][n:]))
        _check(got[r], ref, tol, (op, counts, g))
    assert (got[off[-1]:] == 7.0).all()


def test_strides_and_neighbours():
    """x and out as column slices of wider tensors; what lies beside them stays."""
    m, rng = _m(), np.random.default_rng(5)
    n, k, rows = 37, 80, 5
    w = R.Weight(rng, n, k)
    wide_x = to_dev_bf16(_x(rng, rows, 3 * k))
    wide_y = torch.full((rows, n + 9), 3.0, dtype=torch.bfloat16, device="cuda")
    x = wide_x[:, k:2 * k]
    say("strided gemv")
    m.nvfp4_gemv(x, w.operand(m, torch), rows, n, k, out=wide_y[:, 4:4 + n])
    ref, tol = R.gemv_ref(F.bf16_bits_to_f64(from_dev_bf16(x)), w.dq[0])
    got = F.bf16_bits_to_f64(from_dev_bf16(wide_y))
    _check(got[:, 4:4 + n], ref, tol, "strided")
    assert (got[:, :4] == 3.0).all() and (got[:, 4 + n:] == 3.0).all()


def test_extremes():
    """Zero rows and weights, large and tiny activations, saturated SwiGLU gates."""
    m, rng = _m(), np.random.default_rng(6)
    n, k = 32, 64
    w = R.Weight(rng, 2 * n, k, std=4.0)
    x = F.bf16_bits_to_f64(R.bf16(rng, (6, k)))
    x[0] = 0.0
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -100
    x[3] *= 50.0                                           # gates of some hundreds: exp overflows on one side
    x[4, 1:] = 0.0
    bits = F.bf16_rne(x)
    x = F.bf16_bits_to_f64(bits)
    op = w.operand(m, torch)
    say("extremes")
    y = m.nvfp4_gemv(to_dev_bf16(bits), op, 6, 2 * n, k)
    ref, tol = R.gemv_ref(x, w.dq[0])
    _check(F.bf16_bits_to_f64(from_dev_bf16(y)), ref, tol, "gemv")
    keep = [0, 2, 3, 4, 5]
    h = m.nvfp4_gemv_swiglu(to_dev_bf16(bits[keep]), op, 5, n, k)
    with np.errstate(over="ignore"):
        ref, tol = R.swiglu_ref(x[keep], w.dq[0][:n], w.dq[0][n:])
    _check(F.bf16_bits_to_f64(from_dev_bf16(h)), ref, tol + 2.0 ** -126, "swiglu")


def test_empty():
    m = _m()
    w = R.Weight(np.random.default_rng(1), 16, 32).operand(m, torch)
    x = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    assert m.nvfp4_gemv(x, w, 0, 16, 32).shape == (0, 16)


def test_equal_calls_give_equal_bits():
    m, rng = _m(), np.random.default_rng(9)
    w = R.Weight(rng, 512, 4096).operand(m, torch)
    x = to_dev_bf16(_x(rng, 9, 4096))
    first = m.nvfp4_gemv(x, w, 9, 512, 4096)
    for _ in range(3):
        assert torch.equal(first, m.nvfp4_gemv(x, w, 9, 512, 4096))


@pytest.mark.parametrize("m_rows,n,k", [
    (3, 70, 14336), (9, 300, 8208), (16, 64, 12288),             # long K, few tiles; K no multiple of 64
    (5, 4200, 80), (6, 8200, 96), (11, 24600, 48),               # 263, 513 and 1538 tiles of short K
    (18, 4200, 80), (35, 8208, 144),                             # the same with more than 16 rows
    (20, 8208, 2112), (33, 8224, 4096)])                         # x in registers, 16 rows after 16 rows
def test_tile_counts(m_rows, n, k):
    _dense("gemv", m_rows, n, k, "row", "linear", n + k)


@pytest.mark.parametrize("m_rows,n,k", [(3, 40, 14336), (5, 2104, 80), (9, 4120, 48), (18, 2104, 80), (35, 4104, 144),
                                        (20, 4112, 2112)])
def test_tile_counts_swiglu(m_rows, n, k):
    _dense("swiglu", m_rows, n, k, "row", "linear", n + k)


@pytest.mark.parametrize("block,layout", [("tile", "linear"), ("row", "mfma")])
@pytest.mark.parametrize("m_rows,n,k", [(4, 96, 8192), (18, 4224, 320), (10, 4224, 4160), (20, 8224, 2112)])
def test_tile_counts_of_other_scales(block, layout, m_rows, n, k):
    _dense("gemv", m_rows, n, k, block, layout, n + k)


@pytest.mark.parametrize("m_rows", [1, 2, 5, 20])
@pytest.mark.parametrize("block,layout", [("row", "linear"), ("row", "mfma"), ("tile", "linear")])
@pytest.mark.parametrize("op", ["gemv", "swiglu"])
def test_strided_weight_and_scales_at_any_address(op, block, layout, m_rows):
    """Codes as a column slice of a wider tensor, the scales one byte behind an aligned address."""
    m, rng = _m(), np.random.default_rng(m_rows)
    n, k = 64, 192
    nw = 2 * n if op == "swiglu" else n
    w = R.Weight(rng, nw, k, block, layout)
    wide = torch.randint(0, 256, (nw, k // 2 + 64), dtype=torch.uint8, device="cuda")
    wide[:, 32:32 + k // 2] = torch.from_numpy(w.codes[0]).cuda()
    flat = torch.from_numpy(np.ascontiguousarray(w.scales)).reshape(-1)
    room = torch.full((flat.numel() + 8,), 0x7F, dtype=torch.uint8, device="cuda")      # 0x7F: NaN
    room[1:1 + flat.numel()] = flat.cuda()
    op_w = m.Operand(m.Format.NVFP4, wide[:, 32:32 + k // 2], room[1:1 + flat.numel()].view(w.scales.shape),
                     torch.from_numpy(w.S).cuda(), block=m.Block.TILE if block == "tile" else m.Block.ROW,
                     gs=m.GScale.PER_TENSOR, layout=m.Layout.MFMA if layout == "mfma" else m.Layout.LINEAR)
    x = _x(rng, m_rows, k)
    say(f"strided weight {op} {block} {layout} {m_rows}")
    fn = m.nvfp4_gemv if op == "gemv" else m.nvfp4_gemv_swiglu
    got = F.bf16_bits_to_f64(from_dev_bf16(fn(to_dev_bf16(x), op_w, m_rows, n, k)))
    xv = F.bf16_bits_to_f64(x)
    ref, tol = R.gemv_ref(xv, w.dq[0]) if op == "gemv" else R.swiglu_ref(xv, w.dq[0][:n], w.dq[0][n:])
    _check(got, ref, tol, (op, block, layout, m_rows))


@pytest.mark.parametrize("counts", [[20, 0, 33], [1, 2, 40], [0, 19]])
@pytest.mark.parametrize("k", [80, 192, 2112])
def test_uneven_groups(k, counts):
    """One group far above the average the kernel was chosen by."""
    m, rng = _m(), np.random.default_rng(k + sum(counts))
    n, e = 96, len(counts)
    w = R.Weight(rng, n, k, groups=e)
    rows = sum(counts)
    x = _x(rng, rows, k)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    say(f"uneven groups {k} {counts}")
    got = F.bf16_bits_to_f64(from_dev_bf16(m.nvfp4_gemv(to_dev_bf16(x), w.operand(m, torch), rows, n, k,
                                                        group_row_offsets=torch.from_numpy(off).cuda())))
    for g in range(e):
        r = slice(off[g], off[g + 1])
        ref, tol = R.gemv_ref(F.bf16_bits_to_f64(x)[r], w.dq[g])
        _check(got[r], ref, tol, (k, counts, g))


@pytest.mark.parametrize("m_rows,n,k", [(1, 40, 256), (2, 40, 256), (7, 40, 256), (7, 40, 272), (20, 40, 256)])
def test_infinite_and_nan_rows_stay_by_themselves(m_rows, n, k):
    """A row of x with an infinity or a NaN spoils its own row of y only; so does a row nobody asked for."""
    m, rng = _m(), np.random.default_rng(k + m_rows)
    w = R.Weight(rng, n, k)
    op = w.operand(m, torch)
    x = to_dev_bf16(_x(rng, m_rows + 2, k))
    want = m.nvfp4_gemv(x[:m_rows], op, m_rows, n, k)
    x[m_rows:] = float("nan")
    bad = m_rows - 1
    if m_rows > 1:
        x[bad, 5] = float("inf")
        x[bad, 9] = float("nan")
    say(f"infinite rows {m_rows} {k}")
    got = m.nvfp4_gemv(x[:m_rows], op, m_rows, n, k)
    good = slice(0, bad if m_rows > 1 else 1)
    assert torch.equal(got[good], want[good])
    if m_rows > 1:
        assert got[bad].isnan().all()


@pytest.mark.parametrize("m_rows,k", [(1, 4096), (5, 4096), (6, 4112)])
def test_weights_beyond_four_gibibytes(m_rows, k):
    """The last rows of a large matrix, against the same rows as a matrix of their own."""
    m, rng = _m(), np.random.default_rng(k)
    n, tail = 2_099_200, 64
    w = R.Weight(rng, tail, k)
    codes = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n, k // 16), dtype=torch.uint8, device="cuda")
    codes[-tail:] = torch.from_numpy(w.codes[0]).cuda()
    scales[-tail:] = torch.from_numpy(w.scales[0]).cuda().view(tail, -1)
    assert codes.numel() > 1 << 32
    x = to_dev_bf16(_x(rng, m_rows, k))
    say(f"large weights {m_rows} {k}")
    big = m.nvfp4_gemv(x, m.Operand(m.Format.NVFP4, codes, scales, torch.from_numpy(w.S).cuda(), gs=m.GScale.PER_TENSOR),
                       m_rows, n, k)
    got = F.bf16_bits_to_f64(from_dev_bf16(big[:, -tail:].contiguous()))
    ref, tol = R.gemv_ref(F.bf16_bits_to_f64(from_dev_bf16(x)), w.dq[0])
    _check(got, ref, tol, (m_rows, k))
    assert (big[:, :-tail] == 0).all()
