"""The iteration with the roundings of the library's number formats and no others:
products are exact (64 bits), what is stored is rounded as the header says."""
from __future__ import annotations

import numpy as np

from tests import muon_ref as ref

S = 4096.0      # X, A and B carry it in fp16


def half(x):
    return x.astype(np.float16).astype(np.float64)


def dense(u, steps, coef=(ref.A, ref.B, ref.C), eps=1e-7):
    """A matrix whose smaller side is more than 128 (u as held: bf16 or fp32
    values): X is two fp16 halves and enters products by its high one, A and B are
    one fp16 number.  Returns o before its rounding."""
    a, b, c = coef
    x = u.astype(np.float64)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    f = S / (np.sqrt((x * x).sum()) + eps)
    e = np.floor(np.log2(f))
    r = f / 2.0 ** e
    x = x * 2.0 ** e
    hi = half(x)
    lo = half(x - hi)
    for _ in range(steps):
        A = half(r * r / S * (hi @ hi.T))
        B = half(b * A + c / S * (A @ A))
        x = r / S * (B @ hi) + a * r * (hi + lo)
        hi = half(x)
        lo = half(x - hi)
        r = 1.0
    return (x.T if tall else x) / S


# The figures that the header states, of o before its rounding, by steps.
def stated(shape, steps):
    assert 1 <= steps <= 8
    if min(shape) <= 128:
        return 1.5e-3 if steps <= 5 else 2.5e-3
    return 4e-3 if steps <= 5 else 1.3e-2


KINDS = ["gauss", "power", "power2", "rank1", "rank8", "low", "two", "flat", "geometric"]


def spectrum(rng, shape, kind):
    """A matrix of the given kind of singular values."""
    if kind == "gauss":
        return rng.standard_normal(shape) * 1e-3
    k = min(shape)
    U, _ = np.linalg.qr(rng.standard_normal((shape[0], k)))
    V, _ = np.linalg.qr(rng.standard_normal((shape[1], k)))
    i = np.arange(1, k + 1.0)
    s = {"power": 1 / i, "power2": i ** -2, "rank1": (i == 1) * 1.0, "rank8": np.where(i <= 8, 1.0, 1e-4),
         "low": np.where(i <= 4, 1.0, 1e-3), "two": np.where(i <= 2, 1.0, 0.1), "flat": np.ones(k),
         "geometric": np.geomspace(1, 1e-5, k)}[kind]
    return (U * s) @ V.T
