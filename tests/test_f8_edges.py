"""The 8-bit matrices' calls at the edges of what the header allows, without a GPU:
tests/c/f8_edges.cpp with the host code of their entry points, under the address and
undefined-behaviour sanitizers."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_edges_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("no g++ or HIP headers")
    exe = tmp_path / "f8_edges"
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-fno-omit-frame-pointer",
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__=1",
                    "-isystem", "/opt/rocm/include", os.path.join(ROOT, "tests", "c", "f8_edges.cpp"),
                    os.path.join(ROOT, "zero_sharded_mixed_zero1_amd", "csrc", "f8_api.cpp"), "-o", str(exe)],
                   check=True, capture_output=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1"))
    assert out.returncode == 0, out.stdout[-4000:] + out.stderr[-4000:]
    assert out.stdout.strip().endswith("all ok"), out.stdout[-4000:]
