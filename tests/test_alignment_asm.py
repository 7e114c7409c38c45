"""The alignment that the sources tell the compiler (no GPU): no access is built on a
larger one than the header grants, in the update with 8-bit moments above all, whose
quads lie at any alignment of their elements."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from zero_sharded_mixed_zero1_amd import build

FLAGS = [f for f in build.FLAGS if f not in ("-fPIC", "-shared")]
HIP = [s for s in build.SOURCES if s.endswith(".hip")]


@pytest.mark.parametrize("src", HIP, ids=[os.path.basename(s) for s in HIP])
def test_no_pointer_is_passed_as_better_aligned(src):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = subprocess.run([build.HIPCC, *FLAGS, "--cuda-device-only", "-fsyntax-only", "-Werror=align-mismatch", src],
                         capture_output=True, text=True)
    assert out.returncode == 0, out.stderr[-4000:]


def test_quads_of_the_update_have_their_elements_alignment(tmp_path):
    """master and g at 4 bytes, gradients and parameters at 2; codes and words begin at quads of bytes and words."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "kernels.ll"
    subprocess.run([build.HIPCC, *FLAGS, "--cuda-device-only", "-S", "-emit-llvm", os.path.join(build.HERE, "csrc", "kernels.hip"),
                    "-o", str(out)], check=True, capture_output=True)
    bodies = re.findall(r"^define [^\n]*@(\w*adamw8_kernel\w*)\([^\n]*\{\n(.*?)^\}", out.read_text(), re.S | re.M)
    assert len(bodies) >= 12                               # g or 1 to 4 or any number of slices, flat and over a plan
    most = {"<4 x float>": 4, "<2 x i32>": 2, "i32": 4, "float": 4, "i16": 2, "i8": 1}
    seen = set()
    for name, body in bodies:
        for line in body.splitlines():
            # (what is not quads of floats or non-temporal: descriptors, scalars, codes and words, which lie where the library or the checks put them)
            if not re.search(r"(?:load|store) .*addrspace\(1\)", line) or ("!nontemporal" not in line and "<4 x float>" not in line):
                continue
            got = re.search(r"(?:load|store) (<\d+ x \w+>|\w+)[ ,].*ptr addrspace\(1\) .*align (\d+)", line)
            assert got, f"{name}: {line}"
            seen.add(got[1])
            assert int(got[2]) <= most[got[1]], f"{name}: {line}"
    assert {"<4 x float>", "<2 x i32>"} <= seen, seen
