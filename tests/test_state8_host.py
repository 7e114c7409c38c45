"""Moments in 8 bits without a GPU: sizes, refusals, the arena's layout, and the
reference that the GPU tests compare with against the definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest

import zero_sharded_mixed_zero1_amd as z
from tests import state8_ref as ref

FAKE = 1 << 44


def _einval(f):
    with pytest.raises(z.Zero1Error) as e:
        f()
    assert e.value.name == "ZERO1_EINVAL", e.value
    return e.value.message


@pytest.mark.parametrize("n", [-5, 0, 1, 15, 16, 17, 255, 256, 257, 2048, 2049, 100_003, (1 << 40) - 1])
def test_bytes(n):
    assert z.state8_bytes(n) == ref.size(n)


def test_conversions_refuse():
    enc, dec = z.state8_encode, z.state8_decode
    x, s = FAKE, FAKE + (1 << 30)
    for f in (lambda n, x, s, w, fl=0: enc(x, n, s, w, flags=fl, stream=0), lambda n, x, s, w, fl=0: dec(s, n, x, w, flags=fl, stream=0)):
        assert "n=-1" in _einval(lambda: f(-1, x, s, 0))
        assert "2^34" in _einval(lambda: f((1 << 34) + 1, x, s, 0))
        assert "which" in _einval(lambda: f(10, x, s, 2))
        assert "NULL" in _einval(lambda: f(10, 0, s, 0))
        assert "NULL" in _einval(lambda: f(10, x, 0, 0))
        assert "aligned to its elements" in _einval(lambda: f(10, x + 2, s, 0))
        assert "aligned to its elements" in _einval(lambda: f(10, x + 1, s, 0, z.MV_BF16))
        assert "16-byte" in _einval(lambda: f(10, x, s + 8, 0))
        assert "overlap" in _einval(lambda: f(1000, x, x + 3984, 0))
        assert "overlap" in _einval(lambda: f(1000, x + 1000, x, 1))
        assert "unknown flag" in _einval(lambda: f(10, x, s, 0, 0x1000))
        assert "do not apply" in _einval(lambda: f(10, x, s, 0, z.MV_8BIT))
        assert "do not apply" in _einval(lambda: f(10, x, s, 0, z.STORE_G))


def _piece(n, off, at, m=None, v=None):
    return (n, off, at, at + (1 << 24), m or at + (2 << 24), v or at + (3 << 24))


def test_plan_refuses():
    ps = [_piece(1000, 0, FAKE), _piece(500, 1000, FAKE + (1 << 30))]
    plan = lambda p, fl: z.mta_plan(p, FAKE + (1 << 40), 1 << 20, flags=fl)   # noqa: E731
    assert "exclusive" in _einval(lambda: plan(ps, z.MV_BF16 | z.MV_8BIT))
    assert "16-byte" in _einval(lambda: plan([ps[0], _piece(500, 1000, FAKE + (1 << 30), m=FAKE + (1 << 33) + 8)], z.MV_8BIT))
    assert "16-byte" in _einval(lambda: plan([ps[0], _piece(500, 1000, FAKE + (1 << 30), v=FAKE + (1 << 33) + 4)], z.MV_8BIT))
    # the words behind the codes are part of a buffer: 1008 + 16 bytes
    m = FAKE + (1 << 33)
    assert "overlap" in _einval(lambda: plan([_piece(1000, 0, FAKE, m=m), _piece(500, 1000, FAKE + (1 << 30), m=m + 1008)], z.MV_8BIT))
    # (the same pieces one buffer further apart pass this check and end at the device's)
    with pytest.raises(z.Zero1Error) as e:
        plan([_piece(1000, 0, FAKE, m=m), _piece(500, 1000, FAKE + (1 << 30), m=m + 1024)], z.MV_8BIT)
    assert "overlap" not in e.value.message


def test_flat_step_refuses():
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, max_norm=1.0, step=1)
    step = lambda m, v, fl: z.adamw_step(FAKE, None, 0, 1000, FAKE + (1 << 20), m, v, FAKE + (4 << 20), hp,   # noqa: E731
                                         FAKE + (5 << 20), 1, flags=fl, stream=0)
    a, b = FAKE + (2 << 20), FAKE + (3 << 20)
    assert "exclusive" in _einval(lambda: step(a, b, z.MV_BF16 | z.MV_8BIT))
    assert "16-byte" in _einval(lambda: step(a + 1, b, z.MV_8BIT))
    assert "16-byte" in _einval(lambda: step(a, b + 8, z.MV_8BIT))
    assert "overlap" in _einval(lambda: step(a, a + 1008, z.MV_8BIT))


def test_muon_refuses_8_bit_moments():
    mat = z.matrix(64, 64, param=FAKE, master=FAKE + (1 << 20), m=FAKE + (2 << 20), u=FAKE + (3 << 20))
    assert "unknown flag" in _einval(lambda: z.muon_plan([mat], FAKE + (1 << 30), 1 << 20, flags=z.MV_8BIT))


@pytest.mark.parametrize("S,W", [(1, 1), (1000, 8), (70_001, 3), (842_301_952, 8)])
def test_arena_layout(S, W):
    L = z.arena_plan(S, W, S, 0, S, 0, flags=z.MV_8BIT)
    n = ref.size(S)
    at = sorted([(L.ws, L.ws_bytes), (L.master, 4 * S), (L.m, n), (L.v, n), (L.params, 2 * S)] + [(L.grads[w], 2 * S) for w in range(W)])
    assert all(a + k <= b for (a, k), (b, _) in zip(at, at[1:])) and at[-1][0] + at[-1][1] <= L.total_bytes
    assert L.m % 256 == 0 and L.v % 256 == 0
    assert "exclusive" in _einval(lambda: z.arena_plan(S, W, S, 0, S, 0, flags=z.MV_8BIT | z.MV_BF16))


def _sample(n, seed=0, spread=3.0):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal(n) * np.exp(spread * rng.standard_normal(n))).astype(np.float32)


def test_reference_nearest_is_within_half_a_step():
    x = _sample(20_000)
    codes, words = ref.encode_nearest(x, ref.M)
    y = ref.values(codes, words)
    top = np.repeat(np.abs(np.pad(x, (0, -x.size % 256))).reshape(-1, 256).max(1), 256)[:x.size]
    # half a step: 2^-4 of the value, or 2^-10 units where 2^7 units are at most the block's largest
    assert (np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -17 * top)).all()
    again, words2 = ref.encode_nearest(y.astype(np.float32), ref.M)
    # (rounding up may raise the largest into the next binade: then its own codes differ, its values do not)
    assert np.array_equal(ref.values(again, words2)[np.abs(y) >= 2.0 ** -12 * top], y[np.abs(y) >= 2.0 ** -12 * top])


def test_reference_random_is_floor_plus_share():
    """Against exact rational arithmetic."""
    from fractions import Fraction
    x = _sample(3000, 1)
    bits = np.random.default_rng(2).integers(0, 65536, x.size).astype(np.uint64)
    codes, b = ref.encode_random(x, bits, ref.M)
    for xi, u, c, bi in zip(x, bits, codes, ref.per_element(b, x.size)):
        y = abs(Fraction(float(xi))) / (Fraction(2) ** (int(bi) - 127))
        e = -6
        while Fraction(2) ** (e + 1) <= y:
            e += 1
        step = Fraction(2) ** (e - 3)
        assert Fraction(float(abs(ref.E4M3[c]))) == (y / step + Fraction(int(u), 65536)).__floor__() * step


def test_reference_random_rounding_is_right_on_average():
    """One value, every one of the 65,536 draws: the mean is the value to 2^-17 of a step (and binary32's own bits)."""
    for v in (1.0, 1.03, 3.3, 0.011, 100.0, 2.0 ** -8 * 1.3):
        x = np.full(256, 128.0, np.float32)
        x[:] = v
        x[255] = 128.0
        u = np.arange(65536, dtype=np.uint64)
        y = float(np.float32(v))
        step = 2.0 ** (max(np.floor(np.log2(y)), -6) - 3)
        xs = np.full(65536, v, np.float32)
        xs[255::256] = 128.0
        codes, _ = ref.encode_random(xs, u, ref.M)
        keep = np.arange(65536) % 256 != 255
        want = np.floor(y / step + u / 65536.0) * step
        assert np.array_equal(ref.E4M3[codes][keep], want[keep])
        assert abs(want.mean() - y) <= step * 2.0 ** -16


def test_reference_bits_are_uniform_and_independent():
    n, counts = 256 * 64, 64
    h = np.stack([ref.random_bits(0, np.full(64, c), n) for c in range(counts)]).astype(np.int64)
    for x in (h & 0xFFFF, h >> 16):
        u = x / 65536.0
        # mean of 2^20 draws: 6 sigma of sqrt(1/12 / 2^20)
        assert abs(u.mean() - 0.5) < 6 * (1 / 12 / u.size) ** 0.5
        hist = np.histogram(u, 64, (0, 1))[0]
        e = u.size / 64
        assert ((hist - e) ** 2 / e).sum() < 63 + 6 * (2 * 63) ** 0.5
        for a, b in ((u[1:], u[:-1]), (u[:, 1:], u[:, :-1])):
            assert abs(np.corrcoef(a.ravel(), b.ravel())[0, 1]) < 6 / a.size ** 0.5
    assert abs(np.corrcoef((h & 0xFFFF).ravel(), (h >> 16).ravel())[0, 1]) < 6 / h.size ** 0.5
