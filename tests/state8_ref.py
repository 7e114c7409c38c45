"""Plain numpy reference of moments in 8 bits: the layout, both roundings and
the bits they take, as include/zero1.h states them (no code shared with the
library)."""
from __future__ import annotations

import numpy as np

M, V = 0, 1
BLOCK = 256


def _table():
    t = np.zeros(256, np.float64)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        t[c] = np.nan if (c & 127) == 127 else x
        if c & 128:
            t[c] = -t[c]
    return t


E4M3 = _table()                # what each code stands for
_POSITIVE = E4M3[:127]


def words_at(n):
    return -(-n // 16) * 16


def blocks(n):
    return -(-n // BLOCK)


def size(n):
    return words_at(n) + 4 * blocks(n) if n > 0 else 0


def split(buf, n):
    """Codes and words of a buffer of bytes."""
    return buf[:n], buf[words_at(n):words_at(n) + 4 * blocks(n)].view(np.uint32)


def join(codes, words):
    n = codes.size
    out = np.zeros(size(n), np.uint8)
    out[:n] = codes
    out[words_at(n):] = words.view(np.uint8)
    return out


def per_element(words, n):
    return np.repeat(words, BLOCK)[:n]


def values(codes, words):
    """What the codes stand for before any square, in 64 bits."""
    b = per_element(words & 255, codes.size).astype(np.int64)
    return E4M3[codes] * np.where(b > 0, 2.0 ** (b - 127.0), 0.0)


def decode(codes, words, which):
    with np.errstate(over="ignore"):
        x = values(codes, words).astype(np.float32)
        return x * x if which == V else x


def exponents(x):
    """The exponent byte of each block of fp32 magnitudes."""
    n = x.size
    a = np.zeros(blocks(n) * BLOCK, np.float32)
    a[:n] = np.abs(np.where(np.isfinite(x), x, 0))
    top = a.reshape(-1, BLOCK).max(1)
    return np.maximum((top.view(np.uint32) >> 23).astype(np.int64) - 7, 1)


def _finish(x, code, which):
    code = np.where(per_element(exponents(x), x.size) >= (183 if which == V else 247), np.minimum(code, 0x77), code)
    if which == M:
        code = code | (np.signbit(x).astype(np.int64) << 7)
    else:
        code = np.where(x > 0, np.maximum(code, 1), code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def encode_nearest(x, which):
    """Codes and words of fp32 values (of roots for V), to the nearest, ties to even, from the definition in 64 bits."""
    b = exponents(x)
    y = np.abs(np.where(np.isfinite(x), x, 0)).astype(np.float64) * 2.0 ** (127.0 - per_element(b, x.size))
    hi = np.searchsorted(_POSITIVE, y)                      # the first code at or above y
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - y, y - _POSITIVE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return _finish(x, code, which), b.astype(np.uint32)


def mix(x):
    x = x.astype(np.uint64)
    low = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x6A09E667)) & low
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xBB67AE85)) & low
    return x ^ (x >> np.uint64(16))


def random_bits(first, counts, n):
    """The 32 bits of each of a piece's n elements; first: its place in the shard."""
    low = np.uint64(0xFFFFFFFF)
    starts = (np.arange(blocks(n), dtype=np.uint64) * np.uint64(BLOCK) + np.uint64(first)) & low
    key = mix((mix(starts) + counts.astype(np.uint64)) & low)
    j = np.arange(blocks(n) * BLOCK, dtype=np.uint64) % np.uint64(BLOCK)
    return mix((np.repeat(key, BLOCK) + j) & low)[:n]


def encode_random(x, bits16, which):
    """Codes and exponent bytes of fp32 values rounded by 16 random bits each: floor(|x| / step + u / 65536) steps, in 64
    bits (exact: a binary32 value over a power of two, and 16 bits beside its 24)."""
    b = exponents(x)
    y = np.abs(np.where(np.isfinite(x), x, 0)).astype(np.float64) * 2.0 ** (127.0 - per_element(b, x.size))
    _, e = np.frexp(y)
    e = np.where(y > 0, np.maximum(e - 1, -6), -6)          # the binade; below 2^-6 steps are equal
    k = np.floor(y / 2.0 ** (e - 3.0) + bits16.astype(np.float64) / 65536).astype(np.int64)
    # k steps of 2^(e - 3): 8 to 16 in the binade of e (16: the next one's first), 0 to 8 below
    code = k + (e + 6) * 8
    return _finish(x, code, which), b


def step_words(words, b):
    return ((((words >> np.uint32(8)).astype(np.int64) + 1) & 0xFFFFFF) << 8 | b).astype(np.uint32)


def round_step(m, r, m_words, v_words, first):
    """A piece's new (m codes, m words, v codes, v words) from a step's unrounded m and r and the words before it."""
    bits = random_bits(first, m_words >> np.uint32(8), m.size)
    cm, bm = encode_random(m, bits & np.uint64(0xFFFF), M)
    cv, bv = encode_random(r, bits >> np.uint64(16), V)
    return cm, step_words(m_words, bm), cv, step_words(v_words, bv)
