"""Plain numpy reference of matrices in 8-bit floating point with a power of two
for each block of 128, as include/zero1.h states them (no code shared with the
library)."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def _table(exp_bits, man_bits, bias, inf):
    t = np.zeros(256, np.float64)
    for c in range(256):
        e, f = (c >> man_bits) & ((1 << exp_bits) - 1), c & ((1 << man_bits) - 1)
        x = f * 2.0 ** (1 - bias - man_bits) if e == 0 else ((1 << man_bits) + f) * 2.0 ** (e - bias - man_bits)
        if inf and e == (1 << exp_bits) - 1:
            x = np.inf if f == 0 else np.nan
        if not inf and (c & 127) == 127:
            x = np.nan
        t[c] = -x if c & 128 else x
    return t


E4M3, E5M2 = _table(4, 3, 7, False), _table(5, 2, 15, True)
TABLE = {False: E4M3, True: E5M2}


def ceil(n):
    return -(-n // BLOCK)


def exponents(x, block_rows, e5m2):
    """The exponent byte of each block of fp32 values [rows, cols]."""
    rows, cols = x.shape
    a = np.zeros((-(-rows // block_rows) * block_rows, ceil(cols) * BLOCK), np.float32)
    a[:rows, :cols] = np.abs(np.where(np.isfinite(x), x, 0))
    top = np.ascontiguousarray(a.reshape(-1, block_rows, ceil(cols), BLOCK).max((1, 3)))
    limit = 57344.0 if e5m2 else 448.0
    b = np.ones(top.shape, np.int64)
    with np.errstate(divide="ignore"):
        guess = np.floor(np.log2(top.astype(np.float64) / limit))
    for d in (-1.0, 0.0, 1.0):                              # the least with top <= limit 2^(b - 127)
        e = np.where(top > 0, guess + d, -200)
        fits = top <= limit * 2.0 ** e
        b = np.where(fits & (b == 1) & (e + 127 > 1), (e + 127).astype(np.int64), b)
    return b.astype(np.uint8)


def spread(scales, rows, cols, block_rows):
    """2^(b - 127) of each element."""
    return np.repeat(np.repeat(2.0 ** (scales.astype(np.float64) - 127), block_rows, 0)[:rows], BLOCK, 1)[:, :cols]


def quantize(x, block_rows, e5m2):
    """Codes and exponent bytes, to the nearest, ties to even, from the definition in 64 bits."""
    b = exponents(x, block_rows, e5m2)
    y = np.where(np.isfinite(x), x, 0).astype(np.float64) / spread(b, *x.shape, block_rows)
    t = TABLE[e5m2]
    pos = t[:124] if e5m2 else t[:127]
    a = np.abs(y)
    hi = np.minimum(np.searchsorted(pos, a), pos.size - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo) | (np.signbit(x).astype(np.int64) << 7)
    return code.astype(np.uint8), b


def values(codes, scales, block_rows, e5m2):
    return TABLE[e5m2][codes] * spread(scales, *codes.shape, block_rows)
