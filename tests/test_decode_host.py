"""Device code of the decode step that is plain C++, run on the host."""

import os
import shutil
import subprocess
import sys

import pytest

from tests.util import ROOT

ROCM = "/opt/rocm"


def test_rows_and_requests_agree(tmp_path):
    """The join of split contexts and the append find a row's request by one function, the work units a request's rows
    by another: offsets outside the call must not give a row an owner that has no work units (its place in the
    workspace would never be written)."""
    if shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "requests_check")
    build = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
             "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"),
             "-I", os.path.join(ROOT, "microscaling_quantization_block_amd", "csrc"),
             os.path.join(ROOT, "tests", "sanitize", "requests_check.cpp"), "-o", exe]
    r = subprocess.run(build, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-2000:] + r.stderr[-2000:]


def test_import_without_gpu_support_in_torch():
    """The package imports under a torch built without a GPU, whose private bindings are not there."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import microscaling_quantization_block_amd as m\n"
            "assert m.nvfp4_attention and m.NVFP4Cache\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_launches_without_the_private_bindings(monkeypatch):
    """Where torch lacks the short bindings, the public calls give the device and the stream."""
    import torch
    from microscaling_quantization_block_amd import decode

    class Stream:
        cuda_stream = 0x1234

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream if device == 0 else None)
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    raw_stream, current_device = decode._device_calls()
    assert current_device() == 0 and raw_stream(0) == 0x1234
