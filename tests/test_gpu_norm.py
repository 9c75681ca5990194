"""The norm and its gradient: every output against float64 or, step by step, against the definition's own roundings;
the quantized copies byte for byte against the oracle's quantizers of the kernel's own y."""

import numpy as np
import pytest
import torch

from oracle import formats as F, fp8_blockwise as OB, layout as OL, mxfp8 as OM, nvfp4 as ON
from tests import layer_ref as R
from tests.util import from_dev_bf16, requires_gpu, say, to_dev_bf16, to_np

pytestmark = [pytest.mark.gpu, requires_gpu]

EPS = 1e-6


def _m():
    import microscaling_quantization_block_amd as m
    return m


def _inputs(rng, rows, cols, residual):
    x = F.bf16_rne(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1))))
    return x, F.bf16_rne(1 + 0.1 * rng.standard_normal(cols)), R.bf16(rng, (rows, cols)) if residual else None


def _check_y(n, x, w, r, eps=EPS):
    """rstd within half a step of binary32, h exact, y by the definition's steps from that rstd."""
    h, rstd, y = R.norm_ref(R.f64(x), R.f64(w), eps, None if r is None else R.f64(r))
    got = to_np(n.rstd).astype(np.float64)
    # the mean is off by far less than 2^-40 of itself
    assert (np.abs(got - rstd) <= (R.EPS_F32 + 2.0 ** -40) * rstd + 2.0 ** -150).all()
    if r is not None:
        assert np.array_equal(R.f64(from_dev_bf16(n.h)), h)
    bits = R.norm_y_bits(h, to_np(n.rstd), R.f64(w))
    if n.y is not None:
        assert np.array_equal(from_dev_bf16(n.y), bits)
        tol = (R.EPS_BF16 + 4 * R.EPS_F32) * np.abs(y) + R.TINY_BF16
        assert (np.abs(R.f64(from_dev_bf16(n.y)) - y) <= tol).all()
    return bits


@pytest.mark.parametrize("cols", [8, 24, 128, 136, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 12296, 16384, 32768])
@pytest.mark.parametrize("rows", [1, 7, 33])
@pytest.mark.parametrize("residual", [False, True])
def test_bf16_output(rows, cols, residual):
    m, rng = _m(), np.random.default_rng(rows * cols + residual)
    x, w, r = _inputs(rng, rows, cols, residual)
    say(f"norm {rows}x{cols} residual {residual}")
    n = m.mx_rmsnorm(to_dev_bf16(x), to_dev_bf16(w), EPS, residual=None if r is None else to_dev_bf16(r), with_rstd=True)
    assert (n.h is None) == (r is None) and n.codes is None and n.dq is None
    _check_y(n, x, w, r)


def _quantized(m, fmt, layout, bits):
    """codes, scales (as stored), gscales, dequantized BF16 bits of rows by the oracle."""
    y = R.f64(bits)
    if fmt == m.Format.NVFP4:
        c, s, S = ON.quantize_rowwise(y, "per_row")
        dq = ON.dequantize_bf16(c, s, S, "1x16", "per_row")
    elif fmt == m.Format.MXFP8:
        c, s = OM.quantize_rowwise(y)
        S, dq = None, OM.dequantize_bf16(c, s, "1x32")
    elif fmt == m.Format.FP8_B128:
        c, s = OB.quantize_rows(y)
        S, dq = None, OB.dequantize_bf16(c, s, "1x128")
    else:
        c, s = OB.quantize_rows_f32(y)
        S, dq = None, OB.dequantize_f32s_bf16(c, s, "1x128")
    if layout == m.Layout.MFMA:
        s = OL.linear_to_mfma(s).reshape(s.shape)
    return c, s, S, dq


@pytest.mark.parametrize("fmt", ["MXFP8", "NVFP4", "FP8_B128", "FP8_B128_F32"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (32, 128), (5, 384), (64, 512), (3, 1024), (1, 2048), (9, 2176), (32, 4096),
                                       (2, 8192), (7, 12288), (2, 16384), (3, 32768), (1025, 640), (1056, 1024),
                                       (1024, 2048), (1027, 2304), (1024, 4096)])
@pytest.mark.parametrize("layout", ["LINEAR", "MFMA"])
def test_quantized_output(fmt, rows, cols, layout):
    m, rng = _m(), np.random.default_rng(rows + cols)
    fm, lay = m.Format[fmt], m.Layout[layout]
    if lay == m.Layout.MFMA and (rows % 32 or cols % 128 or fmt.startswith("FP8")):
        return                                             # refused; tested with the other refusals
    x, w, r = _inputs(rng, rows, cols, rows % 2 == 1)
    x[0] = 0                                               # a row of zeros, and in the residual
    if r is not None:
        r[0] = 0
    say(f"norm {fmt} {layout} {rows}x{cols}")
    kw = dict(residual=None if r is None else to_dev_bf16(r), fmt=fm, layout=lay, with_rstd=True)
    xd, wd = to_dev_bf16(x), to_dev_bf16(w)
    n = m.mx_rmsnorm(xd, wd, EPS, with_dq=True, with_y=True, **kw)
    bits = _check_y(n, x, w, r)
    c, s, S, dq = _quantized(m, fm, lay, bits)
    assert np.array_equal(to_np(n.codes), c)
    assert np.array_equal(to_np(n.scales).view(np.uint8), np.ascontiguousarray(s).view(np.uint8).reshape(to_np(n.scales).view(np.uint8).shape))
    if S is not None:
        assert np.array_equal(to_np(n.gscales), S)
    assert np.array_equal(from_dev_bf16(n.dq), dq)
    bare = m.mx_rmsnorm(xd, wd, EPS, **kw)                 # the codes alone
    assert bare.y is None and bare.dq is None
    assert torch.equal(bare.codes, n.codes) and torch.equal(bare.scales, n.scales)


# rows that end inside a lane group, a block's lanes or a wave: odd numbers of blocks
NARROW = [(fmt, "LINEAR", rows, cols) for fmt, widths in (("NVFP4", (16, 48, 144, 272, 1040, 4112)), ("MXFP8", (32, 96, 160, 544, 4128)))
          for cols in widths for rows in (1, 5, 32)] + [("NVFP4", "MFMA", 32, cols) for cols in (64, 192, 576)]


@pytest.mark.parametrize("fmt,layout,rows,cols", NARROW)
def test_quantized_output_of_any_whole_blocks(fmt, layout, rows, cols):
    m, rng = _m(), np.random.default_rng(rows + cols)
    fm, lay = m.Format[fmt], m.Layout[layout]
    x, w, r = _inputs(rng, rows, cols, rows % 2 == 1)
    say(f"norm {fmt} {layout} {rows}x{cols}, whole blocks")
    n = m.mx_rmsnorm(to_dev_bf16(x), to_dev_bf16(w), EPS, residual=None if r is None else to_dev_bf16(r), fmt=fm, layout=lay,
                     with_rstd=True, with_y=True, with_dq=True)
    c, s, S, dq = _quantized(m, fm, lay, _check_y(n, x, w, r))
    assert np.array_equal(to_np(n.codes), c) and np.array_equal(from_dev_bf16(n.dq), dq)
    assert np.array_equal(to_np(n.scales).reshape(-1), np.ascontiguousarray(s).reshape(-1))
    assert S is None or np.array_equal(to_np(n.gscales), S)


def test_bytes_of_the_quantizers():
    """The fused copies are those of the library's own quantizers."""
    m, rng = _m(), np.random.default_rng(5)
    x, w, r = (to_dev_bf16(t) for t in _inputs(rng, 96, 1024, True))
    say("norm against quantizers")
    y = m.mx_rmsnorm(x, w, EPS, residual=r).y
    for fmt, q in ((m.Format.MXFP8, m.mx_quantize), (m.Format.FP8_B128, m.fp8bw_quantize),
                   (m.Format.FP8_B128_F32, m.fp8bw_quantize_f32), (m.Format.NVFP4, m.nvfp4_quantize)):
        n = m.mx_rmsnorm(x, w, EPS, residual=r, fmt=fmt, with_dq=True)
        want = q(y)
        assert torch.equal(n.codes, want[0]) and torch.equal(n.scales, want[1]), fmt
        if fmt == m.Format.NVFP4:
            assert torch.equal(n.gscales, want[2])
        dq = m.mx_dequantize(fmt, n.codes, n.scales, 96, 1024, gscales=n.gscales,
                             gs=m.GScale.PER_ROW if fmt == m.Format.NVFP4 else m.GScale.NONE)
        assert torch.equal(n.dq, dq), fmt


@pytest.mark.parametrize("cols", [128, 512, 640, 2048, 4096])
def test_same_bits_for_any_number_of_rows(cols):
    """One row alone (four waves), a few, and more than a thousand (a wave a row) agree bit for bit."""
    m, rng = _m(), np.random.default_rng(cols)
    x, w, r = (to_dev_bf16(t) for t in _inputs(rng, 1300, cols, True))
    say(f"rows alone and together, {cols}")
    fmts = [m.Format.BF16, m.Format.NVFP4, m.Format.MXFP8]
    for fmt in fmts:
        full = m.mx_rmsnorm(x, w, EPS, residual=r, fmt=fmt, with_rstd=True, with_y=True)
        for lo, hi in ((0, 1), (700, 733), (1299, 1300)):
            part = m.mx_rmsnorm(x[lo:hi], w, EPS, residual=r[lo:hi], fmt=fmt, with_rstd=True, with_y=True)
            for name in ("y", "h", "rstd", "codes", "scales", "gscales"):
                a, b = getattr(full, name), getattr(part, name)
                assert (a is None) == (b is None)
                assert a is None or torch.equal(a[lo:hi], b), (fmt, name, lo)


# from 2048 rows on, 1025 to 4096 columns are a wave a row: whole and partial waves, every format and layout
WAVE_A_ROW = [(fmt, "LINEAR", rows, cols) for rows, cols in ((2048, 2048), (2051, 1152), (2080, 2304), (2049, 4096))
              for fmt in ("MXFP8", "NVFP4", "FP8_B128", "FP8_B128_F32")] + \
             [(fmt, "MFMA", rows, cols) for rows, cols in ((2048, 2048), (2080, 1152), (2112, 2304), (2048, 4096))
              for fmt in ("MXFP8", "NVFP4")]


@pytest.mark.parametrize("fmt,layout,rows,cols", WAVE_A_ROW)
def test_quantized_output_of_a_wave_a_row(fmt, layout, rows, cols):
    """Every byte of a learner's batch against the oracle's quantizers of y."""
    m, rng = _m(), np.random.default_rng(rows + cols)
    fm, lay = m.Format[fmt], m.Layout[layout]
    x, w, r = _inputs(rng, rows, cols, True)
    x[0] = r[0] = x[rows - 1] = r[rows - 1] = 0            # rows of zeros
    say(f"norm {fmt} {layout} {rows}x{cols}, a wave a row")
    kw = dict(residual=to_dev_bf16(r), fmt=fm, layout=lay, with_rstd=True)
    xd, wd = to_dev_bf16(x), to_dev_bf16(w)
    n = m.mx_rmsnorm(xd, wd, EPS, with_y=True, with_dq=True, **kw)
    c, s, S, dq = _quantized(m, fm, lay, _check_y(n, x, w, r))
    assert np.array_equal(to_np(n.codes), c) and np.array_equal(from_dev_bf16(n.dq), dq)
    assert np.array_equal(to_np(n.scales).reshape(-1), np.ascontiguousarray(s).reshape(-1))
    assert S is None or np.array_equal(to_np(n.gscales), S)
    bare = m.mx_rmsnorm(xd, wd, EPS, **kw)
    assert torch.equal(bare.codes, n.codes) and torch.equal(bare.scales, n.scales) and torch.equal(bare.h, n.h)


@pytest.mark.parametrize("cols", [1024, 1152, 2048, 2304, 4096])
@pytest.mark.parametrize("fmt", ["BF16", "MXFP8", "NVFP4", "FP8_B128", "FP8_B128_F32"])
def test_same_bits_below_and_from_2048_rows(cols, fmt):
    """The kernels that share a row among four waves (2047 rows and fewer) and that give it one (2048 and more) agree."""
    m, rng = _m(), np.random.default_rng(cols)
    fm = m.Format[fmt]
    x, w, r = (to_dev_bf16(t) for t in _inputs(rng, 2100, cols, True))
    say(f"norm {fmt} of 2100 rows and fewer, {cols}")
    kw = dict(fmt=fm, with_rstd=True, with_y=True, with_dq=fm != m.Format.BF16)
    full = m.mx_rmsnorm(x, w, EPS, residual=r, **kw)
    for lo, hi in ((0, 1), (0, 2047), (52, 2100), (53, 2100), (2099, 2100)):
        part = m.mx_rmsnorm(x[lo:hi], w, EPS, residual=r[lo:hi], **kw)
        for name, a, b in zip(full._fields, full, part):
            assert (a is None) == (b is None) and (a is None or torch.equal(a[lo:hi], b)), (name, lo, hi)


@pytest.mark.parametrize("rows,cols", [(33000, 128), (8300, 640), (8300, 2048), (8300, 4096), (2000, 4096), (2100, 8192),
                                       (1100, 16384), (600, 32768)])
@pytest.mark.parametrize("fmt", ["BF16", "NVFP4", "FP8_B128_F32"])
def test_more_rows_than_workgroups(rows, cols, fmt):
    """A workgroup walks several rows: they equal the rows in calls of few."""
    m, rng = _m(), np.random.default_rng(rows)
    fm = m.Format[fmt]
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, r = (torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = to_dev_bf16(F.bf16_rne(1 + 0.1 * rng.standard_normal(cols)))
    say(f"norm walks {rows}x{cols} {fmt}")
    kw = dict(fmt=fm, with_rstd=True, with_y=True, with_dq=fm != m.Format.BF16)
    full = m.mx_rmsnorm(x, w, EPS, residual=r, **kw)
    for lo in (0, rows // 2 - 3, rows - 40):
        part = m.mx_rmsnorm(x[lo:lo + 40], w, EPS, residual=r[lo:lo + 40], **kw)
        for a, b in zip(full, part):
            assert (a is None) == (b is None) and (a is None or torch.equal(a[lo:lo + 40], b)), lo


def test_rows_far_apart():
    """Rows beyond 2^31 elements of their matrix, in both directions."""
    m = _m()
    rows, cols = 530_000, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    tail = torch.randn(50, cols, generator=g, device="cuda").to(torch.bfloat16)
    x[-50:] = tail
    w = torch.full((cols,), 1.5, dtype=torch.bfloat16, device="cuda")
    say("far rows")
    n = m.mx_rmsnorm(x, w, EPS, residual=x, h=x, with_rstd=True)
    want = m.mx_rmsnorm(tail, w, EPS, residual=tail, with_rstd=True)
    assert torch.equal(n.y[-50:], want.y) and torch.equal(x[-50:], want.h) and torch.equal(n.rstd[-50:], want.rstd)
    assert not n.y[:1000].any()
    dx, dw = m.mx_rmsnorm_backward(n.y, x, w, n.rstd)
    small, dw2 = m.mx_rmsnorm_backward(want.y, want.h, w, want.rstd)
    assert torch.equal(dx[-50:], small) and not dx[:1000].any()
    # the rows of zeros add nothing; the others' order differs
    bound = 54 * 2 * R.EPS_F32 * (want.y.double() * want.h.double() * want.rstd[:, None]).abs().sum(0)
    assert ((dw - dw2).abs() <= 2 * bound).all()


def test_padded_inputs_and_new_outputs():
    m, rng = _m(), np.random.default_rng(19)
    x, w, r = (to_dev_bf16(t) for t in _inputs(rng, 21, 256, True))
    pad = lambda t: torch.nn.functional.pad(t, (0, 40))[:, :256]
    say("padded inputs")
    a, b = m.mx_rmsnorm(x, w, EPS, residual=r, with_rstd=True), m.mx_rmsnorm(pad(x), w, EPS, residual=pad(r), with_rstd=True)
    assert torch.equal(a.y, b.y) and torch.equal(a.h, b.h) and b.y.is_contiguous() and b.h.is_contiguous()
    for k in range(2):                                     # one row, of any stride
        one = m.mx_rmsnorm(pad(x)[k:k + 1], w, EPS, residual=r[k:k + 1])
        assert torch.equal(one.y, a.y[k:k + 1])
    u, v = (m.mx_rmsnorm_backward(f(x), f(a.h), w, a.rstd, dresidual=f(r)) for f in (lambda t: t, pad))
    assert torch.equal(u[0], v[0]) and torch.equal(u[1], v[1])


def test_strides_and_in_place():
    m, rng = _m(), np.random.default_rng(9)
    rows, cols = 37, 520
    x, w, r = _inputs(rng, rows, cols, True)
    wide = torch.full((rows, cols + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    xd, rd, wd = to_dev_bf16(x), to_dev_bf16(r), to_dev_bf16(w)
    want = m.mx_rmsnorm(xd, wd, EPS, residual=rd)
    wide[:, 8:8 + cols] = xd
    out = torch.full((rows, cols + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    say("strided rows")
    got = m.mx_rmsnorm(wide[:, 8:8 + cols], wd, EPS, residual=rd, h=wide[:, 8:8 + cols], y=out[:, :cols])
    assert torch.equal(got.y, want.y) and torch.equal(got.h, want.h) and got.h.data_ptr() == wide[:, 8:].data_ptr()
    assert (wide[:, :8] == 3).all() and (wide[:, 8 + cols:] == 3).all() and (out[:, cols:] == 5).all()
    r2, x2 = rd.clone(), xd.clone()
    got = m.mx_rmsnorm(x2, wd, EPS, residual=r2, h=r2, y=x2)          # the sum over the residual, y over x
    assert torch.equal(x2, want.y) and torch.equal(r2, want.h)
    # NVFP4 codes with padding between rows
    codes = torch.full((rows, 288), 7, dtype=torch.uint8, device="cuda")
    plain = m.mx_rmsnorm(xd[:, :512].contiguous(), wd[:512], EPS, fmt=m.Format.NVFP4)
    m.mx_rmsnorm(xd[:, :512], wd[:512].contiguous(), EPS, fmt=m.Format.NVFP4, codes=codes[:, :256])
    assert torch.equal(codes[:, :256], plain.codes) and (codes[:, 256:] == 7).all()


@pytest.mark.parametrize("cols", [128, 640, 4096])
def test_magnitudes(cols):
    """Zeros, subnormals, the largest values (whose squares leave binary32), eps 0; spoilt rows leave the others.  Short
    rows of all magnitudes share a wave."""
    m, rng = _m(), np.random.default_rng(4)
    x = rng.standard_normal((8, cols))
    x[1] = 0.0
    x[2] *= 2.0 ** 120
    x[3] *= 2.0 ** -130
    x[4, 0] = 3.3e38
    x[5] *= 2.0 ** -70
    bits, w = F.bf16_rne(x), R.bf16(rng, cols)
    say("norm magnitudes")
    n = m.mx_rmsnorm(to_dev_bf16(bits), to_dev_bf16(w), EPS, with_rstd=True)
    _check_y(n, bits, w, None)
    keep = [0, 2, 4, 5, 6, 7]                              # without eps, rstd of row 3 is beyond binary32
    z = m.mx_rmsnorm(to_dev_bf16(bits[keep]), to_dev_bf16(w), 0.0, with_rstd=True)
    _check_y(z, bits[keep], w, None, 0.0)
    spoilt = bits.copy()
    spoilt[1, 5] = 0x7F80
    spoilt[6, 7] = 0x7FC0
    for fmt in m.Format:
        a = m.mx_rmsnorm(to_dev_bf16(bits), to_dev_bf16(w), EPS, fmt=fmt, with_y=True, with_dq=fmt != m.Format.BF16)
        if fmt != m.Format.BF16:                           # the smallest and largest scales among them
            c, s, S, dq = _quantized(m, fmt, m.Layout.LINEAR, from_dev_bf16(a.y))
            assert np.array_equal(to_np(a.codes), c) and np.array_equal(from_dev_bf16(a.dq), dq)
            assert np.array_equal(to_np(a.scales), s) and (S is None or np.array_equal(to_np(a.gscales), S))
        b = m.mx_rmsnorm(to_dev_bf16(spoilt), to_dev_bf16(w), EPS, fmt=fmt, with_y=True)
        ok = [0, 2, 3, 4, 5, 7]
        assert torch.equal(a.y[ok], b.y[ok]) and torch.isnan(b.y[6]).all() and torch.isnan(b.y[1, 5])
        if a.codes is not None:
            assert torch.equal(a.codes[ok], b.codes[ok]) and torch.equal(a.scales[ok], b.scales[ok])


@pytest.mark.parametrize("eps", [1e-5, 1.1e-12, 0.3, 7e-40])
def test_eps_is_binary64(eps):
    """Rows so small that eps, which binary32 would round by up to 2^-25 of itself or lose, makes rstd."""
    m, rng = _m(), np.random.default_rng(14)
    x = rng.standard_normal((4, 264)) * np.array([0.0, 1e-3, 1e-1, 1.0])[:, None] * eps ** 0.5
    bits, w = F.bf16_rne(x), R.bf16(rng, 264)
    say(f"norm eps {eps}")
    _check_y(m.mx_rmsnorm(to_dev_bf16(bits), to_dev_bf16(w), eps, with_rstd=True), bits, w, None, eps)


# ------------------------------------------------------------------- gradient

def _backward_inputs(rng, rows, cols, dres):
    h = F.bf16_rne(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1))))
    w, dy = F.bf16_rne(1 + 0.1 * rng.standard_normal(cols)), R.bf16(rng, (rows, cols), 1e-3)
    rstd = (1 / np.sqrt((R.f64(h) ** 2).mean(1) + EPS)).astype(np.float32)
    return h, w, dy, rstd, R.bf16(rng, (rows, cols), 1e-3) if dres else None


@pytest.mark.parametrize("cols", [8, 104, 512, 520, 2048, 2064, 4096, 4104, 8192, 8200, 16384, 16392, 32768])
@pytest.mark.parametrize("rows", [1, 3, 130])
@pytest.mark.parametrize("dres", [False, True])
def test_backward(rows, cols, dres):
    m, rng = _m(), np.random.default_rng(rows + cols)
    h, w, dy, rstd, dr = _backward_inputs(rng, rows, cols, dres)
    say(f"norm backward {rows}x{cols} dres {dres}")
    to = to_dev_bf16
    args = (to(dy), to(h), to(w), torch.from_numpy(rstd).cuda())
    drd = None if dr is None else to(dr)
    dx, dw = m.mx_rmsnorm_backward(*args, dresidual=drd)
    ref, wref, tol, wtol = R.norm_backward_ref(R.f64(dy), R.f64(h), R.f64(w), rstd, None if dr is None else R.f64(dr))
    assert (np.abs(R.f64(from_dev_bf16(dx)) - ref) <= tol).all()
    assert (np.abs(to_np(dw) - wref) <= wtol).all()
    again, dw2 = m.mx_rmsnorm_backward(*args, dresidual=drd)
    assert torch.equal(again, dx) and torch.equal(dw2, dw)
    alone, none = m.mx_rmsnorm_backward(*args, dresidual=drd, with_dweight=False)
    assert none is None and torch.equal(alone, dx)


@pytest.mark.parametrize("rows,cols", [(1030, 512), (2500, 136), (5000, 264), (2100, 1032), (1500, 4096), (700, 8192),
                                       (600, 12296), (300, 20000)])
def test_backward_many_rows(rows, cols):
    """More rows than workgroups: each walks several; dw has many partial sums."""
    m, rng = _m(), np.random.default_rng(rows)
    h, w, dy, rstd, dr = _backward_inputs(rng, rows, cols, True)
    say(f"norm backward {rows}x{cols}")
    dx, dw = m.mx_rmsnorm_backward(to_dev_bf16(dy), to_dev_bf16(h), to_dev_bf16(w), torch.from_numpy(rstd).cuda(),
                                   dresidual=to_dev_bf16(dr))
    ref, wref, tol, wtol = R.norm_backward_ref(R.f64(dy), R.f64(h), R.f64(w), rstd, R.f64(dr))
    assert (np.abs(R.f64(from_dev_bf16(dx)) - ref) <= tol).all()
    assert (np.abs(to_np(dw) - wref) <= wtol).all()


def test_backward_against_differences():
    """Central differences of sum(dy y(h, w)) in float64 at the kernel's inputs: the step d leaves d^2 of the third
    derivative and 2^-52 / d of rounding, both below 2^-20 of the gradients' size here."""
    m, rng = _m(), np.random.default_rng(1)
    rows, cols, d = 3, 40, 1e-4
    h, w = R.f64(R.bf16(rng, (rows, cols))), R.f64(F.bf16_rne(1 + 0.1 * rng.standard_normal(cols)))
    dy = R.f64(R.bf16(rng, (rows, cols)))
    loss = lambda a, b: (dy * R.norm_ref(a, b, EPS)[2]).sum()
    gh, gw = np.zeros_like(h), np.zeros_like(w)
    for i in range(rows):
        for j in range(cols):
            e = np.zeros_like(h)
            e[i, j] = d
            gh[i, j] = (loss(h + e, w) - loss(h - e, w)) / (2 * d)
    for j in range(cols):
        e = np.zeros_like(w)
        e[j] = d
        gw[j] = (loss(h, w + e) - loss(h, w - e)) / (2 * d)
    rstd = (1 / np.sqrt((h ** 2).mean(1) + EPS)).astype(np.float32)
    to = lambda a: to_dev_bf16(F.bf16_rne(a))
    say("norm backward against differences")
    dx, dw = m.mx_rmsnorm_backward(to(dy), to(h), to(w), torch.from_numpy(rstd).cuda())
    _, _, tol, wtol = R.norm_backward_ref(dy, h, w, rstd)
    assert (np.abs(R.f64(from_dev_bf16(dx)) - gh) <= tol + 2.0 ** -20 * np.abs(gh).max()).all()
    assert (np.abs(to_np(dw) - gw) <= wtol + 2.0 ** -20 * np.abs(gw).max()).all()


def test_backward_in_place_and_empty():
    m, rng = _m(), np.random.default_rng(2)
    h, w, dy, rstd, dr = _backward_inputs(rng, 50, 264, True)
    hd, wd, dyd, rd, drd = to_dev_bf16(h), to_dev_bf16(w), to_dev_bf16(dy), torch.from_numpy(rstd).cuda(), to_dev_bf16(dr)
    say("norm backward in place")
    want, dw = m.mx_rmsnorm_backward(dyd, hd, wd, rd, dresidual=drd)
    for over in ("dy", "dres"):
        a, b = dyd.clone(), drd.clone()
        ws = torch.full((m.mx_rmsnorm_backward_workspace(50, 264),), 0xFF, dtype=torch.uint8, device="cuda")
        dx, dw2 = m.mx_rmsnorm_backward(a, hd, wd, rd, dresidual=b, dx=a if over == "dy" else b, workspace=ws)
        assert torch.equal(dx, want) and torch.equal(dw2, dw)
    none = torch.empty((0, 264), dtype=torch.bfloat16, device="cuda")
    dx, dw = m.mx_rmsnorm_backward(none, none, wd, rd[:0])
    assert dx.shape == (0, 264) and (dw == 0).all()
    n = m.mx_rmsnorm(none, wd, EPS, residual=none, fmt=m.Format.BF16, with_rstd=True)
    assert n.y.shape == (0, 264)


@pytest.mark.parametrize("cols", [1032, 4096, 8200, 20000])
def test_backward_in_place_wide(cols):
    m, rng = _m(), np.random.default_rng(cols)
    h, w, dy, rstd, dr = _backward_inputs(rng, 9, cols, True)
    hd, wd, rd = to_dev_bf16(h), to_dev_bf16(w), torch.from_numpy(rstd).cuda()
    say(f"norm backward in place {cols}")
    want, dw = m.mx_rmsnorm_backward(to_dev_bf16(dy), hd, wd, rd, dresidual=to_dev_bf16(dr))
    for over in (0, 1):
        a, b = to_dev_bf16(dy), to_dev_bf16(dr)
        dx, dw2 = m.mx_rmsnorm_backward(a, hd, wd, rd, dresidual=b, dx=(a, b)[over])
        assert torch.equal(dx, want) and torch.equal(dw2, dw)


def test_spoilt_rows_of_the_gradient():
    """A NaN in one row's dy: that row and dw, no other row."""
    m, rng = _m(), np.random.default_rng(3)
    h, w, dy, rstd, _ = _backward_inputs(rng, 20, 136, False)
    bad = dy.copy()
    bad[7, 3] = 0x7FC0
    rd = torch.from_numpy(rstd).cuda()
    say("norm backward spoilt row")
    a, _ = m.mx_rmsnorm_backward(to_dev_bf16(dy), to_dev_bf16(h), to_dev_bf16(w), rd)
    b, dw = m.mx_rmsnorm_backward(to_dev_bf16(bad), to_dev_bf16(h), to_dev_bf16(w), rd)
    ok = [i for i in range(20) if i != 7]
    assert torch.equal(a[ok], b[ok]) and torch.isnan(b[7]).all()
    assert torch.isnan(dw[3]) and not torch.isnan(dw[:3]).any()


def test_captured_and_on_another_stream():
    """Forward and backward in a captured graph, replayed with eager work between; the same on a given stream."""
    m, rng = _m(), np.random.default_rng(6)
    x, w, r = (to_dev_bf16(t) for t in _inputs(rng, 70, 1024, True))
    dy = to_dev_bf16(R.bf16(rng, (70, 1024), 1e-3))
    xb, rb, dyb = x.clone(), r.clone(), dy.clone()

    def step(a, b, c, stream=None):
        n = m.mx_rmsnorm(a, w, EPS, residual=b, fmt=m.Format.NVFP4, with_dq=True, with_rstd=True, stream=stream)
        dx, dw = m.mx_rmsnorm_backward(c, n.h, w, n.rstd, dresidual=n.dq, stream=stream)
        return n.codes, n.scales, n.gscales, n.h, dx, dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xb, rb, dyb)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    say("capture norm")
    with torch.cuda.graph(g):
        out = step(xb, rb, dyb)
    other = torch.cuda.Stream()
    for i in range(4):
        say(f"replay norm {i}")
        xb.copy_(x * (i + 1))
        dyb.copy_(dy.roll(i, 0))
        want = step(x * (i + 1), r, dy.roll(i, 0))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        a, c = x * (i + 1), dy.roll(i, 0)
        other.wait_stream(torch.cuda.current_stream())
        got = step(a, r, c, stream=other)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want)), i
