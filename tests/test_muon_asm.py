"""What the source of the products promises about its assembly (no GPU): m0 is
written and read by the loads into LDS only."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from zero_sharded_mixed_zero1_amd import build

SRC = os.path.join(build.HERE, "csrc", "newton_schulz.hip")


def test_nothing_but_the_loads_into_lds_uses_m0(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "newton_schulz.s"
    flags = [f for f in build.FLAGS if f not in ("-fPIC", "-shared")]
    subprocess.run([build.HIPCC, *flags, "--cuda-device-only", "-S", SRC, "-o", str(out)], check=True, capture_output=True)
    code = [line.split(";")[0].split("//")[0].strip() for line in open(out)]
    code = [line for line in code if line]
    uses = [k for k, line in enumerate(code) if re.search(r"\bm0\b", line)]
    assert uses
    for k in uses:
        assert re.fullmatch(r"s_mov_b32 m0, s\d+", code[k]), code[k]
        assert code[k + 1] == "s_nop 0" and code[k + 2].startswith("global_load_lds_dwordx4"), code[k:k + 3]
    assert sum("global_load_lds" in line for line in code) == len(uses)
