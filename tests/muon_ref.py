"""Plain implementations of the Muon step's operators for the tests: momentum
and update one binary32 operation at a time (the library's contract, bit for
bit) and in 64 bits, the Newton-Schulz iteration in 64 bits with a bound on
what the library's roundings may add to it."""
from __future__ import annotations

import numpy as np

A, B, C = 3.4445, -4.7750, 2.0315
U16 = 2.0 ** -11        # half a step of fp16, relative
BF16 = 2.0 ** -8        # half a step of bf16, relative


def widen(h: np.ndarray) -> np.ndarray:
    return (h.astype(np.uint32) << 16).view(np.float32)


def bf16(x: np.ndarray) -> np.ndarray:
    """Bits of the nearest-even bf16 of fp32 values (NaNs quiet)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where((u & 0x7FFFFFFF) > 0x7F800000, ((u >> 16) | 0x40).astype(np.uint16), r)


def momentum32(g, m, mu, nesterov=True):
    """(m, u) in fp32, one operation at a time."""
    mu = np.float32(mu)
    with np.errstate(all="ignore"):
        m = (mu * m) + g
        u = g + (mu * m) if nesterov else m
    return m.astype(np.float32), u.astype(np.float32)


def update32(p, o, lr, wd, scale, decay_first=False):
    eta = np.float32(lr) * np.float32(scale)
    delta = np.float32(1.0 - lr * wd)
    with np.errstate(all="ignore"):
        return (p * delta) - (eta * o) if decay_first else (p - (eta * o)) * delta


def iterate64(u, steps=5, coef=(A, B, C), eps=1e-7):
    """The iteration on one matrix in 64 bits, by its definition."""
    a, b, c = coef
    x = u.astype(np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def iterate_bound(u, steps=5, coef=(A, B, C), eps=1e-7):
    """How far (2-norm) the library's o may be from iterate64 to first order.

    A step maps the singular values s by p(s) = a s + b s^3 + c s^5.  An error
    already in X is multiplied by at most L, the largest divided difference of
    the odd function p over the singular values and their negatives.  Rounding
    A (each entry by at most 2^-11 of itself, so |dA| <= 2^-11 |A| in the
    2-norm of the entries) moves B X by |b dA X| + |c (dA A + A dA) X|, and
    rounding B by |dB X|; X's own halves add 2^-22 |X|, the fp32 sums
    2^-24 sqrt(n) times as much as a term, counted with a further 2^-20 of
    everything.  fp16 has no step smaller than 2^-24, and X carries 2^12: each
    entry of X is off by up to 2^-37 whatever its size (this counts for a u
    that is small beside eps, and so is its o).  At the end o is rounded to
    bf16.  Returns the bound and |o|."""
    a, b, c = coef
    x = u.astype(np.float64)
    s = np.linalg.svd(x, compute_uv=False) / (np.sqrt((x * x).sum()) + eps)
    err = 0.0
    for it in range(steps):
        p = a * s + b * s ** 3 + c * s ** 5
        t, q = np.concatenate([s, -s, [0.0]]), np.concatenate([p, -p, [0.0]])
        d = t[:, None] - t[None, :]
        with np.errstate(all="ignore"):
            div = np.abs((q[:, None] - q[None, :]) / d)
        div[np.abs(d) < 1e-9] = 0.0
        # p' itself, between neighbours as well
        L = max(div.max(), np.abs(a + 3 * b * s ** 2 + 5 * c * s ** 4).max())
        nA, nB = np.linalg.norm(s ** 2), np.linalg.norm(b * s ** 2 + c * s ** 4)
        top = s.max()
        inj = U16 * (abs(b) * nA + 2 * abs(c) * nA * top ** 2 + nB) * top
        inj += (2.0 ** -21 + 2.0 ** -20) * (abs(a) + abs(b) * top ** 2 + abs(c) * top ** 4) * np.linalg.norm(s)
        inj += 2.0 ** -37 * np.sqrt(x.size) * (abs(a) + abs(b) * top ** 2 + abs(c) * top ** 4)
        err = L * err + inj
        s = np.abs(p)
    size = np.linalg.norm(s)
    return err + BF16 * (size + err), size
