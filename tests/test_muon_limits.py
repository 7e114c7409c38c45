"""Sizes at the ends of the Muon plans' range, without a GPU: tests/c/muon_limits.cpp
under the undefined-behaviour sanitizer."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sizes_at_the_ends_of_the_range(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("no g++ or HIP headers")
    exe = tmp_path / "muon_limits"
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=undefined",
                    "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__=1", "-isystem", "/opt/rocm/include",
                    os.path.join(ROOT, "tests", "c", "muon_limits.cpp"),
                    os.path.join(ROOT, "zero_sharded_mixed_zero1_amd", "csrc", "muon_api.cpp"), "-o", str(exe)],
                   check=True, capture_output=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout[-4000:] + out.stderr[-4000:]
    assert out.stdout.strip().endswith("all ok"), out.stdout[-4000:]
