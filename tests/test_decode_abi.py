"""The decode entry points without a GPU: include/mxq_decode.h and the library agree, invalid arguments are refused on
the host with the documented status, and the binding checks what the device reads unvalidated.  Nothing is launched."""

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
NAMES = ("nvfp4_gemv", "nvfp4_gemv_swiglu", "nvfp4_cache_append", "nvfp4_attention", "nvfp4_attention_workspace")


def _lib():
    import microscaling_quantization_block_amd as m
    from microscaling_quantization_block_amd import decode
    sanitized = os.environ.get("MXQ_TEST_SANITIZED_LIBRARY")
    if sanitized:
        m.library_path = sanitized
    if not os.path.exists(m.library_path):
        pytest.skip("libmxq.so not built (run __graft_entry__.build())")
    return m, decode, decode._lib()


def test_header_and_library_agree():
    _, _, L = _lib()
    text = open(os.path.join(ROOT, "include", "mxq_decode.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = re.findall(r"^(?:mxq_status|int64_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert sorted(declared) == sorted(NAMES)
    for n in declared:
        assert hasattr(L, n)


@pytest.mark.parametrize("fn", ["nvfp4_gemv", "nvfp4_gemv_swiglu"])
def test_gemv_rejects_bad_arguments(fn):
    m, d, L = _lib()
    B, G, Lay, Fm = m.Block, m.GScale, m.Layout, m.Format

    def call(x=FAKE, ld_x=64, x_rows=2, M=2, N=32, K=64, y=FAKE, ld_y=32, groups=0, off=None, index=None,
             fmt=Fm.NVFP4, data=0x10000, scales=0x10000, gs=0x10000, block=B.ROW, gmode=G.PER_TENSOR,
             layout=Lay.LINEAR, ld=64, transposed=0):
        w = m._Operand(fmt, data, scales, gs, block, gmode, layout, ld, transposed)
        return getattr(L, fn)(x, ld_x, x_rows, ctypes.byref(w), M, N, K, y, ld_y, groups, off, index, None)

    for kw in (dict(x=None), dict(y=None), dict(data=0), dict(scales=0), dict(gs=0), dict(M=-1), dict(N=-1),
               dict(K=-16), dict(groups=-1), dict(groups=2), dict(x_rows=3), dict(ld_x=56), dict(ld_y=31),
               dict(ld=48), dict(block=B.COL), dict(block=B.NONE), dict(layout=5), dict(x_rows=0, index=FAKE)):
        assert call(**kw) == EINVAL, kw
        assert fn in m.lib().mxq_last_error().decode()
    for kw in (dict(K=40), dict(block=B.TILE, N=24), dict(layout=Lay.MFMA, K=48), dict(layout=Lay.MFMA, N=24)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(x=ODD), dict(ld_x=68), dict(data=0x10008), dict(ld=72), dict(y=ctypes.c_void_p(0x10001)),
               dict(gs=0x10002)):
        assert call(**kw) == EALIGN, kw
    for kw in (dict(fmt=Fm.MXFP8), dict(fmt=Fm.BF16), dict(transposed=1), dict(K=0), dict(gmode=G.PER_ROW),
               dict(block=B.TILE, layout=Lay.MFMA), dict(N=1 << 26, ld_y=1 << 26),
               dict(groups=70000, off=FAKE)):
        assert call(**kw) == EUNSUPPORTED, kw
    assert getattr(L, fn)(FAKE, 64, 2, None, 2, 32, 64, FAKE, 32, 0, None, None, None) == EINVAL
    assert call(M=0, x_rows=0) == 0 and call(N=0) == 0      # nothing to do, nothing launched


def _cache(d, **kw):
    c = dict(k_codes=0x10000, k_scales=0x10000, k_gscales=0x10000, v_codes=0x10000, v_scales=0x10000,
             v_gscales=0x10000, num_pages=4, code_stride=2 * 16 * 64, scale_stride=2 * 16 * 8, gscale_stride=32,
             num_heads=2, page_size=16, head_dim=128)
    c.update(kw)
    return d._Cache(*[c[n] for n, _ in d._Cache._fields_])


BAD_CACHE = [(dict(k_codes=0), EINVAL), (dict(v_scales=0), EINVAL), (dict(k_gscales=0), EINVAL),
             (dict(num_pages=0), EINVAL), (dict(num_pages=-1), EINVAL), (dict(num_heads=0), EINVAL),
             (dict(code_stride=1024), EINVAL), (dict(scale_stride=128), EINVAL), (dict(gscale_stride=16), EINVAL),
             (dict(head_dim=96), EUNSUPPORTED), (dict(head_dim=512), EUNSUPPORTED), (dict(page_size=8), EUNSUPPORTED),
             (dict(page_size=48), EUNSUPPORTED), (dict(page_size=2048), EUNSUPPORTED),
             (dict(k_codes=0x10008), EALIGN), (dict(v_gscales=0x10004), EALIGN), (dict(v_scales=0x10002), EALIGN),
             (dict(code_stride=2 * 16 * 64 + 8), EALIGN), (dict(gscale_stride=34), EALIGN)]


def test_cache_append_rejects_bad_arguments():
    m, d, L = _lib()

    def call(k=FAKE, ks=(256, 128), v=FAKE, vs=(256, 128), tokens=3, cache=(), table=FAKE, ld=4, width=4, lens=FAKE,
             offs=None, n=3, kd=None, vd=None):
        c = ctypes.byref(_cache(d, **dict(cache)))
        return L.nvfp4_cache_append(k, *ks, v, *vs, tokens, c, table, ld, width, lens, offs, n, kd, vd, None)

    for kw, status in BAD_CACHE:
        assert call(cache=kw.items()) == status, kw
    for kw in (dict(k=None), dict(v=None), dict(lens=None), dict(table=None), dict(tokens=-1), dict(n=-1),
               dict(width=-1), dict(ld=3), dict(tokens=4), dict(ks=(-8, 128))):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(k=ODD), dict(vs=(256, 100)), dict(kd=ODD), dict(vd=ODD), dict(lens=ctypes.c_void_p(0x10002))):
        assert call(**kw) == EALIGN, kw
    assert call(tokens=1 << 31, offs=FAKE) == EUNSUPPORTED
    assert call(tokens=1 << 28, offs=FAKE) == EUNSUPPORTED
    assert L.nvfp4_cache_append(FAKE, 256, 128, FAKE, 256, 128, 3, None, FAKE, 4, 4, FAKE, None, 3, None, None,
                                None) == EINVAL
    assert call(tokens=0, n=0) == 0 and call(tokens=0, offs=FAKE) == 0


def test_attention_rejects_bad_arguments():
    m, d, L = _lib()

    def call(q=FAKE, qs=(1024, 128), tokens=3, hq=8, cache=(), table=FAKE, ld=4, width=4, lens=FAKE, offs=None, n=3,
             scale=0.1, window=0, out=FAKE, os_=(1024, 128), lse=None, ws=None, ws_bytes=0):
        c = ctypes.byref(_cache(d, **dict(cache)))
        return L.nvfp4_attention(q, *qs, tokens, hq, c, table, ld, width, lens, offs, n, scale, window, out, *os_,
                                 lse, ws, ws_bytes, None)

    for kw, status in BAD_CACHE:
        assert call(cache=kw.items()) == status, kw
    for kw in (dict(q=None), dict(out=None), dict(lens=None), dict(table=None), dict(tokens=-1), dict(window=-1),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(ld=3), dict(tokens=4), dict(os_=(-8, 8)),
               dict(width=4000, ld=4000), dict(width=4000, ld=4000, ws=FAKE, ws_bytes=100)):
        assert call(**kw) == EINVAL, kw
    assert "workspace" in m.lib().mxq_last_error().decode()
    for kw in (dict(hq=7), dict(hq=0), dict(hq=1)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(q=ODD), dict(out=ODD), dict(qs=(1024, 100)), dict(lse=ctypes.c_void_p(0x10002)),
               dict(width=4000, ld=4000, ws=ODD, ws_bytes=1 << 40)):
        assert call(**kw) == EALIGN, kw
    assert call(tokens=1 << 30, n=5, offs=FAKE) == EUNSUPPORTED
    assert call(tokens=0, n=0) == 0


def test_workspace_follows_the_shapes():
    m, d, L = _lib()
    ws = m.nvfp4_attention_workspace
    assert ws(0, 8, 2, 128, 16, 10, 0, False) == 0
    assert ws(4096, 32, 8, 128, 16, 100, 4096, False) == 0            # enough requests to fill the chip
    assert ws(2, 32, 8, 128, 64, 2048, 2, False) > 0                  # two long contexts are split
    assert ws(2, 32, 8, 128, 64, 2048, 2, True) > 0
    assert ws(2, 32, 8, 128, 64, 1, 2, False) == 0                    # one page: nothing to split
    for bad in ((1 << 40, 32, 8, 128, 64, 2048, 2), (2, 32, 8, 128, 64, 1 << 60, 2), (2, 32, 8, 128, 0, 2048, 2),
                (2, 32, 8, 128, 64, -1, 2), (2, 32, 8, 128, 64, 2048, 1 << 62)):
        assert ws(*bad, False) == 0                                   # the call refuses these


def test_binding_refuses_before_the_library_is_called():
    m, d, L = _lib()
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = m.Operand(m.Format.NVFP4, torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(32, 4, dtype=torch.uint8),
                  torch.ones(1), gs=m.GScale.PER_TENSOR)
    with pytest.raises(TypeError):
        m.nvfp4_gemv(cpu, w, 4, 32, 64)                               # not on a GPU
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    f32 = lambda *s: torch.zeros(s)
    with pytest.raises(ValueError):                                   # a cache of host memory
        m.NVFP4Cache(u8(2, 1, 16, 64), u8(2, 1, 16, 8), f32(2, 1, 16), u8(2, 1, 16, 64), u8(2, 1, 8, 16),
                     f32(2, 1, 16))
    with pytest.raises(TypeError):
        m.NVFP4Cache(None, None, None, None, None, None)
    t = torch.zeros(3, 4, dtype=torch.int32)
    for fn, args in ((m.nvfp4_cache_append, (cpu, cpu)), (m.nvfp4_attention, (cpu,))):
        with pytest.raises(TypeError):
            fn(*args, object(), t, t[:, 0])                           # not a cache


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
                 "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), "-I", csrc,
                 os.path.join(csrc, "api.cpp"), os.path.join(csrc, "api_decode.cpp"),
                 os.path.join(san, "host_stubs.cpp"), os.path.join(san, "host_stubs_decode.cpp"),
                 "-L", os.path.join(rocm, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(rocm, 'lib')}", "-o", lib]
        r = subprocess.run(build, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        env = dict(os.environ)
        env.update(LD_PRELOAD=asan, MXQ_TEST_SANITIZED_LIBRARY=lib,
                   ASAN_OPTIONS="detect_leaks=0:detect_odr_violation=0:halt_on_error=1:abort_on_error=0",
                   UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                            os.path.join(ROOT, "tests", "test_decode_abi.py")],
                           cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
        report = r.stdout[-4000:] + r.stderr[-4000:]
        assert r.returncode == 0, report
        assert "passed" in r.stdout and "ERROR: AddressSanitizer" not in report and "runtime error" not in report
    finally:
        shutil.rmtree(tmp, ignore_errors=True)
