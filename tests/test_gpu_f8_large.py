"""Products of 8-bit matrices by the large tiles, over many blocks of the summed axis and in
every pair of formats: exactly where every sum is a whole number, and random operands
against 64 bits."""
from __future__ import annotations

import numpy as np
import pytest

import zero_sharded_mixed_zero1_amd as z
from tests import f8_ref as ref
from tests.gpu_util import torch_cuda
from tests.test_gpu_f8 import Mat, product, source, whole_numbers
from tests.test_gpu_state8 import bf16_bits, widen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, dev


def in_64_bits(env, va, vb):
    torch, dev = env
    return (torch.from_numpy(va).to(dev) @ torch.from_numpy(vb).to(dev).T.contiguous()).cpu().numpy()


# into bf16: whole tiles of 256 beside bands of 64 rows and of 128, 11 and 17 blocks; whole ones alone; bands of 64 and of 128 alone; tiles of
# 128, and with the summed axis in parts; of 64 over 64 blocks (twice), and in parts.  Into fp32: tiles of 128, from the seventh on in parts, the
# last of 64.
SHAPES = [(4100, 4200, 1300), (4100, 5400, 2100), (5000, 5000, 1300), (1001, 2304, 777), (1500, 4000, 2000), (1500, 4096, 1000),
          (2064, 71, 7077), (2304, 768, 8192), (513, 1100, 8192), (33, 1000, 8192)]


@pytest.mark.parametrize("m,n,k", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
@pytest.mark.parametrize("e5a,e5b", [(True, False), (False, True), (True, True), (False, False)], ids=["e5m2-e4m3", "e4m3-e5m2", "e5m2-e5m2", "e4m3-e4m3"])
def test_many_blocks_of_whole_numbers_are_exact(env, m, n, k, e5a, e5b):
    torch, dev = env
    a, va = whole_numbers(env, m, k, m + k, 1, e5a)
    b, vb = whole_numbers(env, n, k, n + k + 1, 128, e5b)
    want = in_64_bits(env, va, vb).astype(np.float32)      # (whole numbers below 2^24)
    for f32 in (True, False):
        ws = torch.full((max(256, z.f8_product_workspace_bytes(a.m, b.m, z.F32 if f32 else 0)),), 0xFF, dtype=torch.uint8, device=dev)
        got = product(env, a, b, f32, ws=ws)
        assert np.array_equal(got, want if f32 else widen(bf16_bits(want))), f"f32={f32}: {(got != want).sum()} of {got.size}"


@pytest.mark.parametrize("m,n,k", [(2200, 2500, 1500), (1500, 4096, 1000), (2064, 71, 7077), (1001, 2304, 777)],
                         ids=["256", "128", "128 in parts", "256 in bands of 64"])
@pytest.mark.parametrize("e5a", [False, True], ids=["e4m3", "e5m2"])
def test_large_tiles_against_64_bits(env, m, n, k, e5a):
    """Operands as quantize makes them.  Into fp32: k + k / 128 additions, each off by 2^-23 of the sum of magnitudes at
    most.  Into bf16: as many, what eight products lose at most (7 * 2^-10 of the largest: of their magnitudes), and 2^-8 of the result."""
    xa, xb = (source(env, r, k, r + k, True, spread=1.0)[0] for r in (m, n))
    qa, qb = ref.quantize(xa, 1, e5a), ref.quantize(xb, 128, False)
    a, b = Mat(env, m, k, 1, e5a).put(*qa), Mat(env, n, k, 128).put(*qb)
    va, vb = ref.values(*qa, 1, e5a), ref.values(*qb, 128, False)
    want, mag = in_64_bits(env, va, vb), in_64_bits(env, np.abs(va), np.abs(vb))
    got = product(env, a, b, True).astype(np.float64)
    fp32 = (k + k / 128) * 2.0 ** -23
    assert (np.abs(got - want) <= fp32 * mag).all()
    assert np.linalg.norm(got - want) <= 4 * k ** 0.5 * 2.0 ** -23 * np.linalg.norm(mag)
    got = product(env, a, b, False).astype(np.float64)
    assert (np.abs(got - want) <= (fp32 + 7 * 2.0 ** -10) * mag + 2.0 ** -8 * np.abs(got)).all()
    # in the 2-norm: the result's rounding at most, and 1e-4 of it for the sums
    assert np.linalg.norm(got - want) <= (2.0 ** -8 + 1e-4) * np.linalg.norm(want) + 4 * k ** 0.5 * 2.0 ** -23 * np.linalg.norm(mag)
