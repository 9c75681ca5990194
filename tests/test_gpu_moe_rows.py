"""The router, the rows of the experts and the way there and back, against float64 references on the host."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests import layer_ref as R
from tests.util import from_dev_bf16, requires_gpu, say, to_dev_bf16, to_np

pytestmark = [pytest.mark.gpu, requires_gpu]


def _m():
    import microscaling_quantization_block_amd as m
    return m


def _logits(rng, T, E, dtype, kind):
    x = rng.standard_normal((T, E))
    if kind == "ties":                                     # few values, both zeros among them
        x = np.round(x)
        x[::2] *= -1.0
    if kind == "masked":                                   # some experts hidden, one token without any
        x[rng.random((T, E)) < 0.4] = -np.inf
        x[T // 2] = -np.inf
    if kind == "spread":
        x *= 30.0
        x[0] = np.finfo(np.float32).min if dtype == "f32" else -3.38e38      # a mask of the type's lowest value
        x[0, E // 2] = 0.5
    if dtype == "f32":
        x = x.astype(np.float32)
        return x.astype(np.float64), torch.from_numpy(x).cuda()
    b = F.bf16_rne(x)
    return R.f64(b), to_dev_bf16(b)


def _check_rows(got, ids, E):
    offsets, row_token, row_of = R.rows_ref(ids, E)
    assert np.array_equal(to_np(got.offsets), offsets)
    assert np.array_equal(to_np(got.row_of), row_of)
    assert np.array_equal(to_np(got.row_token), row_token)


SIZES = [(1, 1, 1), (3, 5, 2), (64, 16, 16), (65, 17, 3), (100, 60, 4), (64, 128, 8), (200, 128, 8), (1000, 100, 8),
         (33, 200, 6), (70, 256, 9), (20, 256, 17), (300, 300, 8), (64, 512, 10), (90, 512, 64), (40, 1000, 40),
         (130, 1024, 64), (2100, 64, 2), (8200, 8, 2), (9000, 40, 1)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "spread"])
def test_route(T, E, k, dtype, kind):
    m, rng = _m(), np.random.default_rng(T + E + k)
    x, xd = _logits(rng, T, E, dtype, kind)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for renorm in (True, False):
        say(f"route T {T} E {E} k {k} {dtype} {kind} renorm {renorm}")
        r = m.mx_moe_route(xd, k, renormalize=renorm)
        ids, w, tol = R.route_ref(x, k, renorm)
        assert np.array_equal(to_np(r.experts), ids)
        assert (np.abs(to_np(r.weights) - w) <= tol).all()
        _check_rows(r, ids, E)
        d = m.mx_moe_route_backward(torch.from_numpy(dw).cuda(), xd, r.experts, r.weights, renormalize=renorm)
        assert d.dtype == xd.dtype
        ref, dtol = R.route_backward_ref(dw.astype(np.float64), x, ids, w, renorm)
        got = to_np(d).astype(np.float64) if dtype == "f32" else R.f64(from_dev_bf16(d))
        if dtype == "bf16":
            dtol = R.EPS_BF16 * np.abs(ref) + (1 + R.EPS_BF16) * dtol + R.TINY_BF16
        assert (np.abs(got - ref) <= dtol).all()


@pytest.mark.parametrize("T", [5, 300])
def test_route_with_nan_and_infinities(T):
    """A NaN is the largest logit; it, and an infinity, make their token's weights NaN and no other's."""
    m, rng = _m(), np.random.default_rng(7)
    x = rng.standard_normal((T, 40)).astype(np.float32)
    clean = torch.from_numpy(x.copy()).cuda()
    x[1, 7] = np.nan
    x[2, 30] = np.inf
    x[3, 4] = -np.nan
    x[3, 9] = np.inf
    say(f"route NaN {T}")
    xd = torch.from_numpy(x).cuda()
    for renorm in (True, False):
        a, b = m.mx_moe_route(clean, 4, renormalize=renorm), m.mx_moe_route(xd, 4, renormalize=renorm)
        ids, _, _ = R.route_ref(x.astype(np.float64), 4, renorm)
        assert np.array_equal(to_np(b.experts), ids)
        assert ids[1, 0] == 7 and ids[2, 0] == 30 and list(ids[3, :2]) == [4, 9]
        _check_rows(b, ids, 40)
        ok = [t for t in range(T) if t not in (1, 2, 3)]
        assert torch.equal(a.weights[ok], b.weights[ok])
        assert torch.isnan(b.weights[1]).all() and torch.isnan(b.weights[2, 0]) and torch.isnan(b.weights[3]).all()


def test_route_strides_and_given_buffers():
    m, rng = _m(), np.random.default_rng(8)
    wide = torch.from_numpy(rng.standard_normal((150, 77)).astype(np.float32)).cuda()
    x = wide[:, 5:55]
    say("route strides")
    want = m.mx_moe_route(x.contiguous(), 3)
    i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
    ws = torch.full((m.mx_moe_workspace(150, 50, 3),), 0xFF, dtype=torch.uint8, device="cuda")
    got = m.mx_moe_route(x, 3, experts=i32(150, 3), offsets=i32(51), row_token=i32(450), row_of=i32(150, 3), workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dw = torch.randn(150, 3, device="cuda")
    out = torch.full((150, 60), 9.0, device="cuda")
    d = m.mx_moe_route_backward(dw, x, want.experts, want.weights, dlogits=out[:, :50])
    assert torch.equal(d, m.mx_moe_route_backward(dw, x.contiguous(), want.experts, want.weights)) and (out[:, 50:] == 9).all()


def test_route_of_no_tokens():
    m = _m()
    say("no tokens")
    r = m.mx_moe_route(torch.empty((0, 12), device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 13 and r.row_of.shape == (0, 2)
    assert m.mx_moe_sort(r.experts, 12).offsets.tolist() == [0] * 13


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (7, 3, 4), (512, 128, 8), (513, 128, 8), (1000, 1000, 5), (4096, 9, 1),
                                   (4097, 9, 1), (20000, 128, 8), (3000, 1024, 64), (30000, 33, 3)])
def test_sort(T, E, k):
    """Ids outside the experts, repeated ones, experts without tokens and with all of them."""
    m, rng = _m(), np.random.default_rng(T + E)
    for kind in ("any", "one", "outside", "none"):
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        if kind == "one":
            ids[:] = E - 1
        if kind == "outside":
            ids[rng.random((T, k)) < 0.5] = -1
            ids[0, 0], ids[-1, -1] = E, -2147483648
        if kind == "none":
            ids[:] = 2147483647
        say(f"sort T {T} E {E} k {k} {kind}")
        got = m.mx_moe_sort(torch.from_numpy(ids).cuda(), E)
        _check_rows(got, ids, E)


@pytest.mark.parametrize("T,E,k", [(65, 9, 1), (16, 128, 8), (43, 128, 8), (64, 128, 8), (100, 40, 10), (128, 1024, 16),
                                   (2047, 1000, 1), (2048, 3, 1), (256, 128, 8), (2049, 3, 1), (205, 33, 10)])
def test_sort_by_one_workgroup(T, E, k):
    """64 to 2048 slots, one workgroup whose waves have one to four pieces of 64 each, and the first sizes beyond."""
    m, rng = _m(), np.random.default_rng(T + E + k)
    for kind in ("any", "last", "outside"):
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        if kind == "last":
            ids[:] = E - 1
        if kind == "outside":
            ids[rng.random((T, k)) < 0.5] = -1
            ids[0, 0], ids[-1, -1] = E, -2147483648
        say(f"sort by one workgroup T {T} E {E} k {k} {kind}")
        _check_rows(m.mx_moe_sort(torch.from_numpy(ids).cuda(), E), ids, E)


# groups of more tokens than their workgroup routes at once: beyond 16384 tokens of 16 lanes, 4096 of a wave; the last
# pass of a group is a partial one
@pytest.mark.parametrize("T,E,k", [(17000, 16, 2), (40000, 60, 4), (20000, 128, 8), (5000, 200, 6), (4500, 100, 20),
                                   (9000, 512, 10), (4200, 1000, 33)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_in_several_passes(T, E, k, dtype):
    m, rng = _m(), np.random.default_rng(T + E)
    x, xd = _logits(rng, T, E, dtype, "masked")
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    for renorm in (True, False):
        say(f"route in passes T {T} E {E} k {k} {dtype} renorm {renorm}")
        r = m.mx_moe_route(xd, k, renormalize=renorm)
        ids, w, tol = R.route_ref(x, k, renorm)
        assert np.array_equal(to_np(r.experts), ids)
        assert (np.abs(to_np(r.weights) - w) <= tol).all()
        _check_rows(r, ids, E)
        # a token's gradient is the same in a call of few
        d = m.mx_moe_route_backward(dw, xd, r.experts, r.weights, renormalize=renorm)
        for lo, hi in ((0, 40), (T // 2 - 20, T // 2 + 20), (T - 33, T)):
            part = m.mx_moe_route_backward(dw[lo:hi], xd[lo:hi], r.experts[lo:hi], r.weights[lo:hi], renormalize=renorm)
            assert torch.equal(d[lo:hi], part)


def test_sort_of_many_slots():
    """More slots than 256 groups of 65535 hold."""
    m, rng = _m(), np.random.default_rng(3)
    T, E, k = 300_000, 24, 64
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    say("sort of 19 million slots")
    _check_rows(m.mx_moe_sort(torch.from_numpy(ids).cuda(), E), ids, E)


# ------------------------------------------------------------- there and back

def _case(rng, T, k, cols, E=16, missing=0.3):
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < missing] = -1
    ids[0] = -1                                            # a token without rows
    _, _, row_of = R.rows_ref(ids, E)
    return row_of, R.bf16(rng, (T * k, cols)), rng.standard_normal((T, k)).astype(np.float32)


@pytest.mark.parametrize("T,k", [(1, 1), (2, 3), (37, 8), (300, 2), (20, 9), (11, 64)])
@pytest.mark.parametrize("cols", [8, 24, 64, 136, 512, 2048, 2056, 4104])
def test_there_and_back(T, k, cols):
    m, rng = _m(), np.random.default_rng(T * cols + k)
    row_of, rows, w = _case(rng, T, k, cols)
    x, dout = R.bf16(rng, (T, cols)), R.bf16(rng, (T, cols))
    say(f"dispatch and combine T {T} k {k} cols {cols}")
    rd, od, wd = to_dev_bf16(rows), torch.from_numpy(row_of).cuda(), torch.from_numpy(w).cuda()
    M = T * k
    has = row_of >= 0
    for weights in (None, w):
        out = m.mx_moe_combine(rd, od, None if weights is None else wd)
        ref, tol = R.combine_ref(R.f64(rows), row_of, None if weights is None else weights.astype(np.float64))
        assert (np.abs(R.f64(from_dev_bf16(out)) - ref) <= tol).all()
    buf = torch.full((M, cols), 3.0, dtype=torch.bfloat16, device="cuda")
    got = from_dev_bf16(m.mx_moe_dispatch(to_dev_bf16(x), od, out=buf))
    want = np.broadcast_to(F.bf16_rne(np.array([3.0])), (M, cols)).copy()
    tok = np.broadcast_to(np.arange(T)[:, None], (T, k))
    want[row_of[has]] = x[tok[has]]
    assert np.array_equal(got, want)                       # rows of no slot stay
    buf.fill_(3.0)
    dr, dw = m.mx_moe_combine_backward(to_dev_bf16(dout), rd, od, wd, drows=buf)
    want[:] = F.bf16_rne(np.array([3.0]))
    # one binary32 product, then BF16
    prod = (w[..., None] * R.f64(dout)[:, None].astype(np.float32)).astype(np.float32)
    want[row_of[has]] = F.bf16_rne(prod[has].astype(np.float64))
    assert np.array_equal(from_dev_bf16(dr), want)
    y = np.where(has[..., None], R.f64(rows)[np.where(has, row_of, 0)], 0.0)
    t = y * R.f64(dout)[:, None]
    assert (np.abs(to_np(dw) - t.sum(-1)) <= (cols + 1) * 2 * R.EPS_F32 * np.abs(t).sum(-1)).all()
    assert (to_np(dw)[~has] == 0).all()


def test_rows_outside_and_strides():
    """Entries outside the rows are no rows; strided matrices on both sides."""
    m, rng = _m(), np.random.default_rng(12)
    T, k, cols, M = 9, 3, 40, 20
    row_of = rng.permutation(T * k).reshape(T, k).astype(np.int32)           # some are beyond M
    row_of[2, 1], row_of[3, 0] = -5, 2147483647
    ok = (row_of >= 0) & (row_of < M)
    wide = torch.full((M, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    rows = R.bf16(rng, (M, cols))
    wide[:, 8:48] = to_dev_bf16(rows)
    w = rng.standard_normal((T, k)).astype(np.float32)
    od, wd = torch.from_numpy(row_of).cuda(), torch.from_numpy(w).cuda()
    out = torch.full((T, 56), 5.0, dtype=torch.bfloat16, device="cuda")
    say("rows outside")
    m.mx_moe_combine(wide[:, 8:48], od, wd, out=out[:, :40])
    ref, tol = R.combine_ref(R.f64(rows), row_of, w.astype(np.float64))
    assert (np.abs(R.f64(from_dev_bf16(out[:, :40])) - ref) <= tol).all() and (out[:, 40:] == 5).all()
    x = to_dev_bf16(R.bf16(rng, (T, cols)))
    to = torch.full((M, 56), 5.0, dtype=torch.bfloat16, device="cuda")
    m.mx_moe_dispatch(x, od, out=to[:, 8:48])
    named = np.zeros(M, bool)
    for t in range(T):
        for j in range(k):
            if ok[t, j]:
                named[row_of[t, j]] = True
                assert torch.equal(to[row_of[t, j], 8:48], x[t])
    assert (to[:, :8] == 5).all() and (to[:, 48:] == 5).all() and (to[torch.from_numpy(~named).cuda()] == 5).all()
    dr = torch.full((M, 40), 5.0, dtype=torch.bfloat16, device="cuda")
    _, dw = m.mx_moe_combine_backward(x, wide[:, 8:48], od, wd, drows=dr)
    assert (to_np(dw)[~ok] == 0).all() and (dr[torch.from_numpy(~named).cuda()] == 5).all()
    none = m.mx_moe_combine(wide[:0, 8:48], od, wd)
    assert (none == 0).all()


def test_rows_far_apart():
    """Rows beyond 2^31 elements of their matrix."""
    m = _m()
    M, cols, T, k = 530_000, 4096, 40, 3
    rows = torch.zeros((M, cols), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dout = (torch.randn(T, cols, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand(T, k, generator=g, device="cuda")
    row_of = (M - 1 - torch.randperm(T * k, generator=g, device="cuda")).int().view(T, k)
    near = (row_of - (M - T * k)).contiguous()
    say("far rows")
    m.mx_moe_dispatch(x, row_of, out=rows)
    small = m.mx_moe_dispatch(x, near)
    assert torch.equal(rows[-T * k:], small) and not rows[:1000].any()
    assert torch.equal(m.mx_moe_combine(rows, row_of, w), m.mx_moe_combine(small, near, w))
    out = torch.zeros_like(rows)
    _, dw = m.mx_moe_combine_backward(dout, rows, row_of, w, drows=out)
    ds, dw2 = m.mx_moe_combine_backward(dout, small, near, w)
    assert torch.equal(dw, dw2) and torch.equal(out[-T * k:], ds) and not out[:1000].any()


def test_masked_rows_may_hold_anything():
    """A NaN in a row of no slot, and in the rows of a slot that is not there, reaches nothing."""
    m, rng = _m(), np.random.default_rng(13)
    row_of, rows, w = _case(rng, 40, 4, 64)
    od, wd = torch.from_numpy(row_of).cuda(), torch.from_numpy(w).cuda()
    clean = to_dev_bf16(rows)
    spoilt = clean.clone()
    used = torch.zeros(160, dtype=torch.bool, device="cuda")
    used[od[od >= 0].long()] = True
    spoilt[~used] = float("nan")
    dirty = torch.where(od >= 0, wd, torch.full_like(wd, float("nan")))      # weights of missing slots too
    say("spoilt rows")
    assert torch.equal(m.mx_moe_combine(clean, od, wd), m.mx_moe_combine(spoilt, od, dirty))


def test_gradient_against_differences():
    """Logits -> weights -> combined rows: central differences of sum(dout out) in float64 at the same choice, step d: d^2
    of the third derivative and 2^-52 / d of rounding stay below 2^-20 of the largest gradient."""
    m, rng = _m(), np.random.default_rng(21)
    T, E, k, cols, d = 6, 10, 3, 32, 1e-4
    x = rng.standard_normal((T, E)).astype(np.float32)
    rows, dout = R.bf16(rng, (T * k, cols)), R.bf16(rng, (T, cols))
    for renorm in (True, False):
        say(f"router gradient renorm {renorm}")
        xd = torch.from_numpy(x).cuda()
        r = m.mx_moe_route(xd, k, renormalize=renorm)
        ids, row_of = to_np(r.experts), to_np(r.row_of)

        def loss(a):
            p = np.exp(a - a.max(1, keepdims=True))
            g = np.take_along_axis(p, ids, 1)
            w = g / (g if renorm else p).sum(1, keepdims=True)
            return (R.f64(dout) * (R.f64(rows)[row_of] * w[..., None]).sum(1)).sum()

        num = np.zeros((T, E))
        for t in range(T):
            for e in range(E):
                step = np.zeros((T, E))
                step[t, e] = d
                num[t, e] = (loss(x + step) - loss(x - step)) / (2 * d)
        _, dw = m.mx_moe_combine_backward(to_dev_bf16(dout), to_dev_bf16(rows), r.row_of, r.weights)
        dl = to_np(m.mx_moe_route_backward(dw, xd, r.experts, r.weights, renormalize=renorm))
        _, w64, _ = R.route_ref(x.astype(np.float64), k, renorm)
        dw64 = (R.f64(rows)[row_of] * R.f64(dout)[:, None]).sum(-1)
        _, tol = R.route_backward_ref(dw64, x.astype(np.float64), ids, w64, renorm)
        # dw itself: cols additions of products of this size
        tol = tol + (cols + 1) * 2 * R.EPS_F32 * (np.abs(R.f64(rows)[row_of]) * np.abs(R.f64(dout))[:, None]).sum(-1).max()
        assert (np.abs(dl - num) <= tol + 2.0 ** -20 * np.abs(num).max()).all()


def test_rows_of_the_products():
    """offsets and row_token as the grouped products take them, some experts missing: rows of no expert are untouched, the
    others are the dispatched rows times their expert's matrix."""
    m, rng = _m(), np.random.default_rng(31)
    from tests import decode_ref as D
    T, E, k, K, N = 50, 6, 2, 64, 32
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[:, 4] = -np.inf
    logits[7, 1:] = -np.inf                                # one expert is left for this token
    x = to_dev_bf16(R.bf16(rng, (T, K)))
    w = D.Weight(rng, N, K, groups=E)
    r = m.mx_moe_route(torch.from_numpy(logits).cuda(), k)
    n = int(r.offsets[-1])
    assert n == T * k - 1
    y = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    say("grouped products on routed rows")
    m.nvfp4_gemv(x, w.operand(m, torch), T * k, N, K, out=y, group_row_offsets=r.offsets, x_row_index=r.row_token)
    assert (y[n:] == 7).all()
    rows = R.f64(from_dev_bf16(m.mx_moe_dispatch(x, r.row_of)))
    off = to_np(r.offsets)
    for e in range(E):
        ref, tol = D.gemv_ref(rows[off[e]:off[e + 1]], w.dq[e])
        assert (np.abs(R.f64(from_dev_bf16(y[off[e]:off[e + 1]])) - ref) <= tol).all()
    q = m.nvfp4_quantize(x, gs=m.GScale.PER_ROW)
    A = m.Operand(m.Format.NVFP4, *q, gs=m.GScale.PER_ROW)
    g = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    m.mx_gemm(A, w.operand(m, torch), T * k, N, K, out=g, group_row_offsets=r.offsets, a_row_index=r.row_token, a_rows=T)
    assert (g[n:] == 7).all()
    xq = R.f64(from_dev_bf16(m.mx_dequantize(m.Format.NVFP4, *q[:2], T, K, gscales=q[2], gs=m.GScale.PER_ROW)))
    tok = to_np(r.row_token)
    for e in range(E):
        ref = xq[tok[off[e]:off[e + 1]]] @ w.dq[e].T
        got = R.f64(from_dev_bf16(g[off[e]:off[e + 1]]))
        # x was rounded to BF16 once more for this reference
        size = np.abs(xq[tok[off[e]:off[e + 1]]]) @ np.abs(w.dq[e]).T
        assert (np.abs(got - ref) <= R.EPS_BF16 * np.abs(ref) + 1.1 * R.EPS_BF16 * size).all()


def test_captured_and_on_two_streams():
    """Router, dispatch, combine and their gradients captured; replays with eager work between; two streams at once."""
    m, rng = _m(), np.random.default_rng(41)
    T, E, k, cols = 300, 24, 4, 72
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    x, dout = (to_dev_bf16(R.bf16(rng, (T, cols))) for _ in range(2))

    def step(lg, a, g, stream=None):
        r = m.mx_moe_route(lg, k, renormalize=False, stream=stream)
        rows = m.mx_moe_dispatch(a, r.row_of, stream=stream)
        out = m.mx_moe_combine(rows, r.row_of, r.weights, stream=stream)
        dr, dw = m.mx_moe_combine_backward(g, rows, r.row_of, r.weights, stream=stream)
        dl = m.mx_moe_route_backward(dw, lg, r.experts, r.weights, renormalize=False, stream=stream)
        return (*r, rows, out, dr, dw, dl, m.mx_moe_combine(dr, r.row_of, stream=stream))

    lb, xb = logits.clone(), x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(lb, xb, dout)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    say("capture")
    with torch.cuda.graph(g):
        out = step(lb, xb, dout)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(4):
        say(f"replay {i}")
        a, b = logits.roll(i, 1).contiguous(), x.roll(i, 0).contiguous()
        lb.copy_(a)
        xb.copy_(b)
        want = step(a, b, dout)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want)), i
        c = logits.roll(-i, 1).contiguous()
        other = step(c, b, dout)
        torch.cuda.synchronize()
        got = [step(p, b, dout, stream=s) for p, s in zip((a, c), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got[0], want)), i
        assert all(torch.equal(u, v) for u, v in zip(got[1], other)), i
