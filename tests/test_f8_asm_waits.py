"""What the ring of stages in LDS needs of the 8-bit products' assembly (no GPU): loads
into LDS overwrite a stage that waves have just read, and the compiler does not know
that they write there.  So on every path through every kernel no LDS read may be on
its way at a barrier, after which another wave's loads may overwrite what it reads;
and in the kernels of few rows, where a wave's ring is its own and nothing else
comes between, at a load into LDS."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from zero_sharded_mixed_zero1_amd import build

SRC = os.path.join(build.HERE, "csrc", "f8_product.hip")


def kernels(text):
    """Each kernel's instructions (labels end in a colon), by name."""
    names = re.findall(r"^\s*\.amdhsa_kernel (\S+)", text, re.M)
    lines = [line.split(";")[0].split("//")[0].strip() for line in text.splitlines()]
    found = {}
    for name in names:
        begin = lines.index(name + ":")
        end = next(k for k in range(begin, len(lines)) if lines[k].startswith(".Lfunc_end"))
        found[name] = [x for x in lines[begin + 1:end] if x and (not x.startswith(".") or x.endswith(":"))]
    return found


def reads_on_their_way(code):
    """Of each instruction, how many LDS reads may still be on their way when it begins, the most over all paths to it (at most 64)."""
    place = {x[:-1]: k for k, x in enumerate(code) if x.endswith(":")}
    state, todo = {0: 0}, [0]
    while todo:
        k = todo.pop()
        x, n = code[k], state[k]
        if x.startswith(("ds_read", "ds_load", "ds_bpermute", "ds_permute", "ds_swizzle")):
            n = min(n + 1, 64)
        elif x.startswith("s_waitcnt"):
            got = re.search(r"lgkmcnt\((\d+)\)", x)
            assert got or "vmcnt" in x, x
            # (reads return in order; scalar loads count with them but may overtake, so only a wait for all of them counts)
            n = 0 if got and int(got[1]) == 0 else n
        nexts = [k + 1]
        if x.startswith(("s_branch", "s_cbranch")):
            nexts = [place[x.split()[1]]] + ([k + 1] if x.startswith("s_cbranch") else [])
        elif x.startswith("s_endpgm"):
            nexts = []
        assert not x.startswith(("s_setpc", "s_swappc", "s_call")), x
        for j in nexts:
            if j < len(code) and state.get(j, -1) < n:
                state[j] = n
                todo.append(j)
    return state


def broken(code, thin):
    """The instructions that must not begin while reads are on their way, and do."""
    state = reads_on_their_way(code)
    watched = [k for k, x in enumerate(code) if x.startswith("s_barrier") or (thin and x.startswith("global_load_lds"))]
    assert watched
    return [(k, code[k], state[k]) for k in watched if state.get(k, 0)]


@pytest.fixture(scope="module")
def found(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("asm") / "f8_product.s"
    flags = [f for f in build.FLAGS if f not in ("-fPIC", "-shared")]
    subprocess.run([build.HIPCC, *flags, "--cuda-device-only", "-S", SRC, "-o", str(out)], check=True, capture_output=True)
    return kernels(out.read_text())


def test_no_read_is_on_its_way_where_its_stage_may_be_overwritten(found):
    rings = {name: code for name, code in found.items() if any("global_load_lds" in x for x in code)}
    assert sum("thin_kernel" in n for n in rings) >= 24 and sum("tile_kernel" in n for n in rings) >= 24 and sum("big_kernel" in n for n in rings) >= 4
    for name, code in rings.items():
        assert any(x.startswith(("ds_read", "ds_load")) for x in code)
        assert broken(code, "thin_kernel" in name) == [], name


def test_a_missing_wait_is_found(found):
    """The same code with the waits for LDS before its barriers taken out one by one: each is missed where reads came before."""
    name = next(n for n in found if "big_kernel" in n)
    code = found[name]
    barriers = [k for k, x in enumerate(code) if x.startswith("s_barrier")]
    missed = 0
    for k in barriers:
        waits = [j for j in range(max(0, k - 3), k) if re.search(r"lgkmcnt\(0\)", code[j])]
        cut = [x for j, x in enumerate(code) if j not in waits]
        missed += bool(waits) and bool(broken(cut, False))
    assert missed >= len(barriers) // 3
