"""The steps around a layer's products without a GPU: include/mxq_layer.h and the library agree, invalid arguments are
refused on the host with the documented status, and the binding checks what the device reads unvalidated.  Nothing is
launched."""

import ctypes
import os
import re
import shutil
import subprocess
import sys
import tempfile

import pytest
import torch

from tests.util import ROOT

FAKE = ctypes.c_void_p(0x10000)       # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)
EINVAL, ESHAPE, EALIGN, EUNSUPPORTED = 1, 2, 3, 4
NAMES = ["mx_rmsnorm", "mx_rmsnorm_backward", "mx_rmsnorm_backward_workspace", "mx_moe_route", "mx_moe_route_backward",
         "mx_moe_sort", "mx_moe_workspace", "mx_moe_dispatch", "mx_moe_combine", "mx_moe_combine_backward",
         "nvfp4_rope_append"]


def _lib():
    import microscaling_quantization_block_amd as m
    from microscaling_quantization_block_amd import layer
    sanitized = os.environ.get("MXQ_TEST_SANITIZED_LIBRARY")
    if sanitized:
        m.library_path = sanitized
    if not os.path.exists(m.library_path):
        pytest.skip("libmxq.so not built (run __graft_entry__.build())")
    return m, layer._lib()


def test_header_and_library_agree():
    m, L = _lib()
    text = open(os.path.join(ROOT, "include", "mxq_layer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = re.findall(r"^(?:mxq_status|int64_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert sorted(declared) == sorted(NAMES)
    for n in declared:
        assert hasattr(L, n) and hasattr(m, n) and n in m.__all__


def test_norm_rejects_bad_arguments():
    m, L = _lib()
    Fm, Lay = m.Format, m.Layout

    def call(x=FAKE, ld_x=256, r=None, ld_r=256, w=FAKE, rows=32, cols=256, eps=1e-6, h=None, ld_h=256, y=FAKE, ld_y=256,
             rstd=None, fmt=Fm.BF16, layout=Lay.LINEAR, codes=None, ld_c=256, scales=None, gs=None, dq=None, ld_dq=256):
        return L.mx_rmsnorm(x, ld_x, r, ld_r, w, rows, cols, eps, h, ld_h, y, ld_y, rstd, fmt, layout, codes, ld_c, scales,
                            gs, dq, ld_dq, None)

    fp8 = dict(fmt=Fm.MXFP8, codes=FAKE, scales=FAKE)
    nv = dict(fmt=Fm.NVFP4, codes=FAKE, scales=FAKE, gs=FAKE)
    f32s = dict(fmt=Fm.FP8_B128_F32, codes=FAKE, scales=FAKE)
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(rows=-1), dict(cols=-8), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(ld_x=248), dict(ld_y=248), dict(h=FAKE),
               dict(r=FAKE, ld_r=248), dict(r=FAKE, h=FAKE, ld_h=248), dict(fmt=9), dict(fmt=-1), dict(layout=2),
               dict(codes=FAKE), dict(scales=FAKE), dict(gs=FAKE), dict(dq=FAKE), dict(fp8, codes=None),
               dict(fp8, scales=None), dict(fp8, gs=FAKE), dict(nv, gs=None), dict(fp8, ld_c=240), dict(nv, ld_c=112),
               dict(fp8, dq=FAKE, ld_dq=248)):
        assert call(**kw) == EINVAL, kw
        assert "mx_rmsnorm" in m.lib().mxq_last_error().decode()
    for kw in (dict(cols=252), dict(fp8, cols=240), dict(nv, cols=248), dict(f32s, cols=192), dict(fp8, layout=1, rows=31),
               dict(fp8, layout=1, cols=96), dict(nv, layout=1, cols=96)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(x=ODD), dict(w=ODD), dict(y=ODD), dict(ld_x=260), dict(ld_y=260), dict(r=ODD), dict(r=FAKE, ld_r=260),
               dict(r=FAKE, h=ODD), dict(rstd=ctypes.c_void_p(0x10002)), dict(fp8, codes=ODD), dict(fp8, ld_c=264),
               dict(nv, gs=ctypes.c_void_p(0x10002)), dict(f32s, scales=ctypes.c_void_p(0x10002)), dict(fp8, dq=ODD),
               dict(fp8, dq=FAKE, ld_dq=260)):
        assert call(**kw) == EALIGN, kw
    for kw in (dict(cols=32776, ld_x=32776, ld_y=32776), dict(rows=1 << 31), dict(f32s, layout=1),
               dict(fmt=Fm.FP8_B128, codes=FAKE, scales=FAKE, layout=1), dict(layout=1)):
        assert call(**kw) == EUNSUPPORTED, kw
    assert call(rows=0, x=None, y=None) == 0 and call(cols=0, x=None) == 0      # nothing to do, nothing launched


def test_norm_takes_nvfp4_codes_of_any_whole_blocks():
    """NVFP4 rows are 8 bytes a block, so a stride of 8 bytes is enough, as in nvfp4_quantize; the FP8 formats need 16.
    The values' matrix is checked behind the codes: its status says that the codes passed."""
    m, L = _lib()

    def call(fmt, cols, ld_c):
        nv = fmt == m.Format.NVFP4
        return L.mx_rmsnorm(FAKE, cols, None, 0, FAKE, 4, cols, 1e-6, None, 0, None, 0, None, fmt, 0, FAKE, ld_c, FAKE,
                            FAKE if nv else None, FAKE, cols - 8, None)

    for cols in (16, 32, 48, 144, 272, 4112):
        assert call(m.Format.NVFP4, cols, cols // 2) == EINVAL and "dq" in m.lib().mxq_last_error().decode(), cols
        assert call(m.Format.NVFP4, cols, cols // 2 + 4) == EALIGN, cols
    for cols in (32, 96, 160):
        assert call(m.Format.MXFP8, cols, cols) == EINVAL and call(m.Format.MXFP8, cols, cols + 8) == EALIGN, cols


def test_norm_backward_rejects_bad_arguments():
    m, L = _lib()
    big, need = 1 << 40, m.mx_rmsnorm_backward_workspace(5, 64)

    def call(dy=FAKE, ld_dy=64, h=FAKE, ld_h=64, w=FAKE, rstd=FAKE, dr=None, ld_dr=64, rows=5, cols=64, dx=FAKE, ld_dx=64,
             dw=FAKE, ws=FAKE, ws_bytes=big):
        return L.mx_rmsnorm_backward(dy, ld_dy, h, ld_h, w, rstd, dr, ld_dr, rows, cols, dx, ld_dx, dw, ws, ws_bytes, None)

    for kw in (dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(rows=-1), dict(cols=-8),
               dict(ld_dy=56), dict(ld_h=56), dict(ld_dx=56), dict(dr=FAKE, ld_dr=56), dict(ws=None),
               dict(ws_bytes=need - 1)):
        assert call(**kw) == EINVAL, kw
    assert "workspace" in m.lib().mxq_last_error().decode()
    for kw in (dict(dy=ODD), dict(h=ODD), dict(w=ODD), dict(dx=ODD), dict(dr=ODD), dict(ld_dy=68), dict(dw=ODD), dict(ws=ODD),
               dict(rstd=ctypes.c_void_p(0x10002))):
        assert call(**kw) == EALIGN, kw
    assert call(cols=60) == ESHAPE and call(cols=32776, ld_dy=32776, ld_h=32776, ld_dx=32776) == EUNSUPPORTED
    assert call(rows=1 << 31) == EUNSUPPORTED
    assert call(rows=0, dw=None, ws=None) == 0 and call(cols=0) == 0
    ws = m.mx_rmsnorm_backward_workspace
    assert need > 0 and ws(0, 64) == 0 and ws(-1, 64) == 0 and ws(1 << 40, 64) == 0 and ws(5, 1 << 20) == 0


def test_norm_binding_refuses_before_the_library_is_called():
    m, _ = _lib()
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    for bad in (x, None, x[0]):
        with pytest.raises(TypeError):
            m.mx_rmsnorm(bad, w)                               # not on a GPU, not a matrix
        with pytest.raises(TypeError):
            m.mx_rmsnorm_backward(bad, x, w, torch.zeros(4))


def test_route_and_sort_reject_bad_arguments():
    m, L = _lib()
    big, two = 1 << 40, ctypes.c_void_p(0x10002)

    def route(x=FAKE, f32=1, ld=16, T=100, E=16, k=4, renorm=1, ids=FAKE, w=FAKE, off=FAKE, tok=FAKE, row=FAKE, ws=FAKE,
              n=big):
        return L.mx_moe_route(x, f32, ld, T, E, k, renorm, ids, w, off, tok, row, ws, n, None)

    def sort(ids=FAKE, T=5000, E=16, k=4, off=FAKE, tok=FAKE, row=FAKE, ws=FAKE, n=big):
        return L.mx_moe_sort(ids, T, E, k, off, tok, row, ws, n, None)

    for kw in (dict(x=None), dict(w=None), dict(ids=None), dict(off=None), dict(tok=None), dict(row=None), dict(T=-1),
               dict(E=0), dict(k=0), dict(k=65, E=100, ld=100), dict(ld=15), dict(ws=None), dict(n=127)):
        assert route(**kw) == EINVAL, kw
    for kw in (dict(ids=None), dict(off=None), dict(tok=None), dict(row=None), dict(T=-1), dict(E=0), dict(k=0), dict(k=65),
               dict(ws=None), dict(n=100)):
        assert sort(**kw) == EINVAL, kw
        assert "mx_moe_sort" in m.lib().mxq_last_error().decode()
    assert route(k=17) == ESHAPE
    for kw in (dict(x=two), dict(f32=0, x=ctypes.c_void_p(0x10001)), dict(w=two), dict(ids=two), dict(off=two), dict(ws=ODD)):
        assert route(**kw) == EALIGN, kw
    for kw in (dict(ids=two), dict(tok=two), dict(row=two), dict(ws=ODD)):
        assert sort(**kw) == EALIGN, kw
    for kw in (dict(E=1025, ld=1025), dict(T=1 << 24), dict(T=(1 << 24) - 1, k=5), dict(T=1 << 20, k=64, E=64, ld=64),
               dict(ld=1 << 31)):
        assert route(**kw) == EUNSUPPORTED, kw
    for kw in (dict(E=1025), dict(T=1 << 24), dict(T=(1 << 24) - 1, k=5)):
        assert sort(**kw) == EUNSUPPORTED, kw
    ws = m.mx_moe_workspace
    assert ws(0, 16, 4) == 0 and ws(1, 16, 4) == 0 and ws(100, 16, 4) > 0 and ws(-1, 16, 4) == 0 and ws(1 << 30, 16, 4) == 0
    assert ws(100, 0, 4) == 0 and ws(100, 16, 0) == 0 and ws(100, 1 << 20, 4) == 0


def test_route_backward_rejects_bad_arguments():
    m, L = _lib()
    two = ctypes.c_void_p(0x10002)

    def call(dw=FAKE, x=FAKE, f32=1, ld=16, T=9, E=16, k=4, ids=FAKE, w=FAKE, d=FAKE, ld_d=16):
        return L.mx_moe_route_backward(dw, x, f32, ld, T, E, k, 1, ids, w, d, ld_d, None)

    for kw in (dict(dw=None), dict(x=None), dict(ids=None), dict(w=None), dict(d=None), dict(ld=15), dict(ld_d=15),
               dict(T=-1), dict(E=0), dict(k=0)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(dw=two), dict(x=two), dict(ids=two), dict(w=two), dict(d=two)):
        assert call(**kw) == EALIGN, kw
    assert call(k=17) == ESHAPE and call(E=2000, ld=2000, ld_d=2000) == EUNSUPPORTED and call(T=0, x=None) == 0


def test_rows_calls_reject_bad_arguments():
    m, L = _lib()
    two = ctypes.c_void_p(0x10002)

    def dispatch(x=FAKE, ld=64, T=5, cols=64, row=FAKE, k=2, rows=FAKE, ld_r=64, M=10):
        return L.mx_moe_dispatch(x, ld, T, cols, row, k, rows, ld_r, M, None)

    def combine(rows=FAKE, ld_r=64, M=10, row=FAKE, w=FAKE, T=5, cols=64, k=2, out=FAKE, ld=64):
        return L.mx_moe_combine(rows, ld_r, M, row, w, T, cols, k, out, ld, None)

    def backward(g=FAKE, ld=64, rows=FAKE, ld_r=64, M=10, row=FAKE, w=FAKE, T=5, cols=64, k=2, dr=FAKE, ld_dr=64, dw=FAKE):
        return L.mx_moe_combine_backward(g, ld, rows, ld_r, M, row, w, T, cols, k, dr, ld_dr, dw, None)

    for fn in (dispatch, combine, backward):
        for kw in (dict(row=None), dict(rows=None), dict(T=-1), dict(cols=-8), dict(k=0), dict(k=65), dict(M=-1), dict(ld=56),
                   dict(ld_r=56)):
            assert fn(**kw) == EINVAL, (fn, kw)
        for kw in (dict(rows=ODD), dict(ld=68), dict(ld_r=68), dict(row=two)):
            assert fn(**kw) == EALIGN, (fn, kw)
        assert fn(cols=60) == ESHAPE
        for kw in (dict(T=1 << 24), dict(T=(1 << 24) - 1, k=5), dict(T=1 << 20, k=64), dict(cols=1 << 26, ld=1 << 26, ld_r=1 << 26),
                   dict(M=1 << 31)):
            assert fn(**kw) == EUNSUPPORTED, (fn, kw)
        assert fn(T=0, row=None) == 0
    assert dispatch(x=None) == EINVAL and combine(out=None) == EINVAL and dispatch(x=ODD) == EALIGN
    for kw in (dict(g=None), dict(w=None), dict(dr=None), dict(dw=None), dict(ld_dr=56)):
        assert backward(**kw) == EINVAL, kw
    for kw in (dict(g=ODD), dict(dr=ODD), dict(w=two), dict(dw=two), dict(ld_dr=68)):
        assert backward(**kw) == EALIGN, kw
    assert combine(w=two) == EALIGN and dispatch(M=0) == 0 and dispatch(cols=0) == 0


def test_slots_fill_a_32_bit_grid_at_most():
    """A workgroup of 256 lanes takes four slots: 2^26 - 4 slots are 2^32 - 256 lanes, one more slot is a workgroup more.
    A misaligned array stops the calls that pass the limit before anything is launched."""
    m, L = _lib()
    two, ws = ctypes.c_void_p(0x10002), 1 << 40
    calls = {
        "sort": lambda T, k: L.mx_moe_sort(two, T, 64, k, FAKE, FAKE, FAKE, FAKE, ws, None),
        "route": lambda T, k: L.mx_moe_route(FAKE, 1, 64, T, 64, k, 1, two, FAKE, FAKE, FAKE, FAKE, FAKE, ws, None),
        "route_backward": lambda T, k: L.mx_moe_route_backward(two, FAKE, 1, 64, T, 64, k, 1, FAKE, FAKE, FAKE, 64, None),
        "dispatch": lambda T, k: L.mx_moe_dispatch(FAKE, 64, T, 64, two, k, FAKE, 64, 10, None),
        "combine": lambda T, k: L.mx_moe_combine(FAKE, 64, 10, two, FAKE, T, 64, k, FAKE, 64, None),
        "combine_backward": lambda T, k: L.mx_moe_combine_backward(FAKE, 64, FAKE, 64, 10, two, FAKE, T, 64, k, FAKE, 64, FAKE,
                                                                   None),
    }
    most = (1 << 26) - 4
    for name, call in calls.items():
        for T, k in (((1 << 24) - 1, 4), (1 << 20, 63)):       # the limit itself, and below
            assert T * k <= most and call(T, k) == EALIGN, (name, T, k)
        # 2^26 - 3, 2^26 - 2 twice, 2^26 - 1, 2^26
        for T, k in ((1813753, 37), (1082401, 62), (2164802, 31), (22369621, 3), (1 << 20, 64)):
            assert T * k > most and call(T, k) == EUNSUPPORTED, (name, T, k)
        assert "slots" in m.lib().mxq_last_error().decode()


def test_moe_binding_refuses_before_the_library_is_called():
    m, _ = _lib()
    x, i = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: m.mx_moe_route(x, 2), lambda: m.mx_moe_sort(i, 4), lambda: m.mx_moe_dispatch(x, i),
                 lambda: m.mx_moe_combine(x, i), lambda: m.mx_moe_combine_backward(x, x, i, x),
                 lambda: m.mx_moe_route_backward(x, x, i, x), lambda: m.mx_moe_route(None, 2)):
        with pytest.raises(TypeError):
            call()                                             # not on a GPU


def test_rope_append_rejects_bad_arguments():
    m, L = _lib()
    from microscaling_quantization_block_amd import decode as d
    from tests.test_decode_abi import BAD_CACHE, _cache

    def call(q=FAKE, qs=(1024, 128), hq=8, k=FAKE, ks=(256, 128), v=FAKE, vs=(256, 128), tokens=3, cache=(), table=FAKE, ld=4,
             width=4, lens=FAKE, offs=None, n=3, freq=FAKE, rot=128, inter=0, factor=1.0, out=FAKE, os_=(1024, 128), kd=None,
             vd=None):
        c = ctypes.byref(_cache(d, **dict(cache)))
        return L.nvfp4_rope_append(q, *qs, hq, k, *ks, v, *vs, tokens, c, table, ld, width, lens, offs, n, freq, rot, inter,
                                   factor, out, *os_, kd, vd, None)

    for kw, status in BAD_CACHE:
        assert call(cache=kw.items()) == status, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(freq=None), dict(lens=None), dict(table=None),
               dict(tokens=-1), dict(n=-1), dict(width=-1), dict(ld=3), dict(tokens=4), dict(ks=(-8, 128)), dict(hq=0),
               dict(hq=32768), dict(factor=float("nan")), dict(factor=float("inf"))):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(rot=-16)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(q=ODD), dict(k=ODD), dict(out=ODD), dict(vs=(256, 100)), dict(qs=(1020, 128)), dict(os_=(1024, 100)),
               dict(kd=ODD), dict(vd=ODD), dict(freq=ctypes.c_void_p(0x10002))):
        assert call(**kw) == EALIGN, kw
    assert call(tokens=1 << 25, offs=FAKE) == EUNSUPPORTED and call(tokens=1 << 31, offs=FAKE) == EUNSUPPORTED
    assert call(tokens=0, n=0) == 0 and call(tokens=0, offs=FAKE) == 0


def _runtime(name):
    out = subprocess.run(["g++", f"-print-file-name={name}"], capture_output=True, text=True).stdout.strip()
    return out if os.path.isabs(out) and os.path.exists(out) else None


def test_validation_under_asan_and_ubsan():
    """The host code built with g++ as a host-only library whose launchers are stubs; this file reruns against it
    with the sanitizer runtime preloaded.  No GPU code is built or run."""
    if os.environ.get("MXQ_TEST_SANITIZED_LIBRARY"):
        pytest.skip("inner run")
    rocm = "/opt/rocm"
    if shutil.which("g++") is None or not os.path.isdir(os.path.join(rocm, "include", "hip")):
        pytest.skip("needs g++ and the ROCm headers")
    asan = _runtime("libasan.so")
    if asan is None:
        pytest.skip("libasan not found")
    tmp = tempfile.mkdtemp(prefix="mxq_asan_")
    try:
        lib = os.path.join(tmp, "libmxq_host_asan.so")
        csrc = os.path.join(ROOT, "microscaling_quantization_block_amd", "csrc")
        san = os.path.join(ROOT, "tests", "sanitize")
        build = ["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-fsanitize=address,undefined",
                 "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                 "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), "-I", csrc]
        build += [os.path.join(csrc, f) for f in ("api.cpp", "api_decode.cpp", "api_layer.cpp")]
        build += [os.path.join(san, f) for f in ("host_stubs.cpp", "host_stubs_decode.cpp", "host_stubs_layer.cpp")]
        build += ["-L", os.path.join(rocm, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(rocm, 'lib')}", "-o", lib]
        r = subprocess.run(build, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        env = dict(os.environ)
        env.update(LD_PRELOAD=asan, MXQ_TEST_SANITIZED_LIBRARY=lib,
                   ASAN_OPTIONS="detect_leaks=0:detect_odr_violation=0:halt_on_error=1:abort_on_error=0",
                   UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                            os.path.join(ROOT, "tests", "test_layer_abi.py")],
                           cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
        report = r.stdout[-4000:] + r.stderr[-4000:]
        assert r.returncode == 0, report
        assert "passed" in r.stdout and "ERROR: AddressSanitizer" not in report and "runtime error" not in report
    finally:
        shutil.rmtree(tmp, ignore_errors=True)
