"""8-bit matrices without a GPU: refusals, and the reference that the GPU tests
compare with against its own definition."""
from __future__ import annotations

import weakref

import numpy as np
import pytest

import zero_sharded_mixed_zero1_amd as z
from tests import f8_ref as ref

FAKE = 1 << 44


def _einval(f):
    with pytest.raises(z.Zero1Error) as e:
        f()
    assert e.value.name == "ZERO1_EINVAL", e.value
    return e.value.message


def _m(rows, cols, at=FAKE, **kw):
    codes, scales = kw.pop("codes", at), kw.pop("scales", at + (1 << 36))
    return z.f8_matrix(rows, cols, codes, scales, **kw)


BAD = [
    (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(cols=-1), "cols"), (dict(cols=(1 << 23) + 1), "cols"),
    (dict(block_rows=64), "block_rows"), (dict(block_rows=0), "block_rows"), (dict(flags=1), "unknown flag"),
    (dict(ld=256), "ld="), (dict(ld=392), "ld="), (dict(ld=-384), "ld="), (dict(ld=1 << 25), "ld="),
    (dict(ld_scales=2), "ld_scales"), (dict(ld_scales=6), "ld_scales"), (dict(ld_scales=-4), "ld_scales"),
    (dict(codes=0), "NULL"), (dict(scales=0), "NULL"), (dict(codes=FAKE + 8), "16-byte"), (dict(scales=FAKE + (1 << 36) + 2), "4-byte"),
]


@pytest.mark.parametrize("change,word", BAD, ids=[f"{list(c)[0]}={list(c.values())[0]}" for c, _ in BAD])
def test_matrices_are_refused(change, word):
    shape = dict(rows=100, cols=300)
    m = _m(**{**shape, **change})
    other = _m(50, change.get("cols", 300) if 0 <= change.get("cols", 300) <= 1 << 23 else 300, FAKE + (1 << 40))
    assert word in _einval(lambda: z.f8_product(m, other, FAKE + (1 << 42), stream=0))
    assert word in _einval(lambda: z.f8_product(other, m, FAKE + (1 << 42), stream=0))
    assert word in _einval(lambda: z.f8_quantize(FAKE + (1 << 42), m.rows, m.cols, q=m, stream=0))
    assert word in _einval(lambda: z.f8_quantize(FAKE + (1 << 42), max(m.cols, 0), max(m.rows, 0), qt=m, stream=0)) or m.rows < 0 or m.cols < 0
    assert z.f8_product_workspace_bytes(m, other) == 0


def test_quantize_refuses():
    q, qt, src = _m(100, 300), _m(300, 100, FAKE + (1 << 40)), FAKE + (1 << 42)
    f = lambda s=src, r=100, c=300, q=q, qt=qt, **kw: z.f8_quantize(s, r, c, q=q, qt=qt, stream=0, **kw)   # noqa: E731
    assert "both NULL" in _einval(lambda: f(q=None, qt=None))
    assert ">= 0" in _einval(lambda: f(r=-1))
    assert "q is 100 x 300" in _einval(lambda: f(r=101))
    assert "qt is 300 x 100" in _einval(lambda: f(q=None, c=301))
    assert "ld=299" in _einval(lambda: f(ld=299))
    assert "src is NULL" in _einval(lambda: f(s=0))
    assert "aligned to its elements" in _einval(lambda: f(s=src + 1))
    assert "aligned to its elements" in _einval(lambda: f(s=src + 2, flags=z.F32))
    assert "unknown flag" in _einval(lambda: f(flags=z.E5M2))
    assert "q.codes and src" in _einval(lambda: f(s=FAKE + 38_398))
    assert "q.scales and src" in _einval(lambda: f(s=FAKE + (1 << 36)))
    assert "q.codes and qt.codes" in _einval(lambda: f(qt=_m(300, 100, FAKE, scales=FAKE + (1 << 40))))
    assert "q.scales and qt.scales" in _einval(lambda: f(qt=_m(300, 100, FAKE + (1 << 40), scales=FAKE + (1 << 36) + 396)))
    many = z.f8_matrix(1 << 30, 1 << 12, 1 << 45, 1 << 47)
    assert "2^23" in _einval(lambda: z.f8_quantize(1 << 50, 1 << 30, 1 << 12, q=many, stream=0))


def test_product_refuses():
    a, b, d = _m(100, 300), _m(50, 300, FAKE + (1 << 40)), FAKE + (1 << 42)
    f = lambda a=a, b=b, d=d, **kw: z.f8_product(a, b, d, stream=0, **kw)   # noqa: E731
    assert "columns" in _einval(lambda: f(b=_m(50, 301, FAKE + (1 << 40))))
    assert "ldd=49" in _einval(lambda: f(ldd=49))
    assert "d is NULL" in _einval(lambda: f(d=0))
    assert "aligned to its elements" in _einval(lambda: f(d=d + 1))
    assert "aligned to its elements" in _einval(lambda: f(d=d + 2, flags=z.F32))
    assert "unknown flag" in _einval(lambda: f(flags=0x10))
    tall = z.f8_matrix(1 << 30, 128, 1 << 45, 1 << 47)
    assert "2^21" in _einval(lambda: f(a=_m(1, 128), b=tall, d=1 << 50))
    assert "2^21" in _einval(lambda: f(a=tall, b=_m(1, 128), d=1 << 50))
    for at in (FAKE + 38_399, FAKE + (1 << 36) + 396, FAKE + (1 << 40), FAKE + (1 << 40) + (1 << 36)):
        assert "d and" in _einval(lambda: f(d=at // 2 * 2))


def test_reference_rounds_within_half_a_step():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((130, 300)) * np.exp(4 * rng.standard_normal((130, 300)))).astype(np.float32)
    for e5m2, half, low, limit in ((False, 2.0 ** -4, 2.0 ** -17, 448.0), (True, 2.0 ** -3, 2.0 ** -31, 57344.0)):
        for block in (1, 128):
            codes, b = ref.quantize(x, block, e5m2)
            y = ref.values(codes, b, block, e5m2)
            top = np.abs(np.pad(x, ((0, -130 % block), (0, 84)))).reshape(-1, block, 3, 128).max((1, 3)).astype(np.float64)
            assert (top <= limit * 2.0 ** (b - 127.0)).all() and (top > limit / 2 * 2.0 ** (b - 127.0)).all()
            tops = np.repeat(np.repeat(top, block, 0)[:130], 128, 1)[:, :300]
            assert (np.abs(y - x) <= np.maximum(half * np.abs(x), low * tops)).all()


def test_reference_scales_at_the_borders():
    x = np.array([[448.0], [449.0], [np.nextafter(np.float32(448), np.float32(500))], [0.0], [2.0 ** -149], [1.75], [224.0], [224.1]], np.float32)
    assert ref.exponents(x, 1, False)[:, 0].tolist() == [127, 128, 128, 1, 1, 119, 126, 127]


class _Tensor:   # what the binding asks of a tensor
    is_cuda = True

    def data_ptr(self):
        return FAKE


def test_a_matrix_keeps_its_tensors():
    codes, scales = _Tensor(), _Tensor()
    alive = weakref.ref(codes)
    m = z.f8_matrix(128, 128, codes, scales)
    del codes, scales
    assert alive() is not None and m.codes == FAKE
    del m
    assert alive() is None
