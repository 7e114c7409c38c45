"""What products into bf16 lose in their sums, as include/zero1.h states it: of eight
neighbouring columns the matrix cores cut each product toward zero to a multiple of
2^(E - 13), E the largest sum of two codes' exponents among the eight.  Held to that
on every tile shape: where the sums cancel, by the worst case; on random operands,
with the result's own rounding out of the way, by what such cuts lose of them."""
from __future__ import annotations

import numpy as np
import pytest

import zero_sharded_mixed_zero1_amd as z
from tests import f8_ref as ref
from tests.gpu_util import torch_cuda
from tests.test_gpu_f8 import Mat, product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, dev


def exponent(codes, e5m2):
    """Codes' exponents; one below the smallest normal value counts as that."""
    field = (codes.astype(np.int64) >> (2 if e5m2 else 3)) & (31 if e5m2 else 15)
    return np.maximum(field, 1) - (15 if e5m2 else 7)


class Sums:
    """One row of a against b's rows in 64 bits: exact sums, those of the cut products, the sums of magnitudes, and the most
    that seven cuts in each group can take."""

    def __init__(self, ca, sa, e5a, cb, sb, e5b):
        p = ref.TABLE[e5a][ca][None] * ref.TABLE[e5b][cb]
        e = np.where(p != 0, exponent(ca, e5a)[None] + exponent(cb, e5b), -999).reshape(cb.shape[0], -1, 8).max(2)
        q = np.repeat(2.0 ** (e - 13.0), 8, 1)
        scale = np.repeat(2.0 ** (sa.astype(np.float64)[None] + sb.astype(np.float64) - 254.0), 128, 1)
        self.exact, self.cut = (p * scale).sum(1), (np.trunc(p / q) * q * scale).sum(1)
        self.magnitude, self.most = (np.abs(p) * scale).sum(1), (7 * q * scale)[:, ::8].sum(1)


def product_of_one_row(env, m, row, b, e5a, f32):
    """d's rows where all m of a are alike: they have to be alike too."""
    a = Mat(env, m, b.cols, 1, e5a).put(np.repeat(row[0][None], m, 0), np.repeat(row[1][None], m, 0))
    d = product(env, a, b, f32)
    bits = d.view(np.uint32)
    assert (bits == bits[:1]).all()
    return d[0].astype(np.float64)


# a few rows; tiles of 64, and with the summed axis in parts; of 128, and in parts; of 256 in bands of 64 and of 128 rows; whole ones
SHAPES = [(1, 300, 1408), (20, 300, 1408), (64, 300, 1408), (40, 300, 2432), (1500, 2304, 640), (2064, 71, 7168), (300, 8000, 1408),
          (2200, 2500, 1536), (4096, 4096, 1408)]
IDS = ["x".join(map(str, s)) for s in SHAPES]


def additions(k):
    """At most so many fp32 additions make a sum: one a group of eight, one an instruction, the parts' (16)."""
    return k / 8 + k / 64 + 16


@pytest.mark.parametrize("m,n,k", SHAPES, ids=IDS)
@pytest.mark.parametrize("e5a", [False, True], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("below", [False, True], ids=["normal", "below the smallest normal"])
def test_sums_that_cancel_lose_no_more_than_the_groups_do(env, m, n, k, e5a, below):
    """In each group of eight one product is by far the largest, and the next group's takes it away.  The others are whole
    multiples of 2^-18 (e5m2: 2^-25) and below 2^5, or below 2^-3 where the largest has a code below the smallest normal one: sums
    of them hold in 64 bits, and into fp32 within its additions."""
    rng = np.random.default_rng(m + k)
    ta, tb = ref.TABLE[e5a], ref.TABLE[False]
    code = lambda t, v: int(np.flatnonzero((t == v) & (np.signbit(t) == (v < 0)))[0])   # noqa: E731
    top = 2.0 ** -4 if below else 4.0
    small_a, small_b = (np.flatnonzero(np.isfinite(t) & (np.abs(t) < top)) for t in (ta, tb))
    ca, cb = rng.choice(small_a, k).astype(np.uint8), rng.choice(small_b, (n, k)).astype(np.uint8)
    at = np.arange(k // 8) * 8 + rng.integers(0, 8, k // 8)
    # the largest: 2^8 * 2^8, or the least code there is times 2^8
    ca[at] = code(ta, ta[1] if below else 256.0)
    cb[:, at[0::2]], cb[:, at[1::2]] = code(tb, 256.0), code(tb, -256.0)
    sa, sb = np.full(k // 128, 127, np.uint8), np.full((n, k // 128), 127, np.uint8)
    s = Sums(ca, sa, e5a, cb, sb, False)
    b = Mat(env, n, k, 1).put(cb, sb)
    fp32 = additions(k) * 2.0 ** -23 * s.magnitude
    got = product_of_one_row(env, m, (ca, sa), b, e5a, False)
    assert (np.abs(got - s.exact) <= s.most + fp32 + 2.0 ** -8 * np.abs(got)).all()
    assert np.linalg.norm(got - s.exact) <= np.linalg.norm(s.cut - s.exact) + np.linalg.norm(fp32) + 2.0 ** -8 * np.linalg.norm(got)
    got = product_of_one_row(env, m, (ca, sa), b, e5a, True)
    assert (np.abs(got - s.exact) <= k * 2.0 ** -23 * s.magnitude).all()       # (an addition a product)


@pytest.mark.parametrize("m,n,k", SHAPES, ids=IDS)
@pytest.mark.parametrize("e5a,e5b", [(False, False), (True, False), (False, True)], ids=["e4m3-e4m3", "e5m2-e4m3", "e4m3-e5m2"])
def test_sums_of_random_operands_before_their_rounding(env, m, n, k, e5a, e5b):
    """Operands as quantize makes them.  The last four blocks take each sum away again, a code at a time: what is left is below
    2^-12 of it, so that bf16's rounding of that shows the sum's own error."""
    rng = np.random.default_rng(m + n)
    main = k - 512
    xa, xb = (rng.standard_normal((r, main)) * np.exp(rng.standard_normal((r, main))) for r in (1, n))
    ca, cb = np.zeros(k, np.uint8), np.zeros((n, k), np.uint8)
    sa, sb = np.full(k // 128, 127, np.uint8), np.full((n, k // 128), 127, np.uint8)
    (qa, ea), (qb, eb) = ref.quantize(xa.astype(np.float32), 1, e5a), ref.quantize(xb.astype(np.float32), 1, e5b)
    ca[:main], sa[:main // 128], cb[:, :main], sb[:, :main // 128] = qa[0], ea[0], qb, eb
    result = Sums(ca, sa, e5a, cb, sb, e5b).exact
    ca[main::128] = 0x3C if e5a else 0x38                  # 1
    left = result.copy()
    for block in range(main // 128, k // 128):
        q, e = ref.quantize(-left.astype(np.float32)[:, None], 1, e5b)
        cb[:, 128 * block], sb[:, block] = q[:, 0], e[:, 0]
        left += ref.values(q, e, 1, e5b)[:, 0]
    s = Sums(ca, sa, e5a, cb, sb, e5b)
    assert np.linalg.norm(left) <= 2.0 ** -12 * np.linalg.norm(result)
    got = product_of_one_row(env, m, (ca, sa), Mat(env, n, k, 1, e5b).put(cb, sb), e5a, False)
    off = got - s.exact
    assert (np.abs(off) <= s.most + additions(k) * 2.0 ** -23 * s.magnitude + 2.0 ** -8 * np.abs(got)).all()
    # in the 2-norm: what the cuts take, and the additions' roundings at random (four times the square root of their number)
    rounding = 4 * additions(k) ** 0.5 * 2.0 ** -23 * np.linalg.norm(s.magnitude) + 2.0 ** -8 * np.linalg.norm(got)
    assert np.linalg.norm(off) <= np.linalg.norm(s.cut - s.exact) + rounding
    # the figure that the documents give: cuts computed in 64 bits as above take 1e-5 to 8e-5 of normal operands spread by factors up to e^2
    assert np.linalg.norm(off) <= 1e-4 * np.linalg.norm(result) + rounding
