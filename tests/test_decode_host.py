"""Device code of the decode step that is plain C++, run on the host."""

import os
import shutil
import subprocess

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
