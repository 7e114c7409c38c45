"""What o is before its rounding to bf16, on the GPU, against the iteration in 64
bits: inputs at the ends of the formats' ranges and the figures that the header
states."""
from __future__ import annotations

import numpy as np
import pytest

from tests import muon_ref as ref
from tests.test_gpu_muon import Steps, env  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("u_f32", [False, True])
@pytest.mark.parametrize("size", [1.0, 1e-20, 1e-30])
def test_parts_of_the_gram_sum_that_hold_only_zeros(env, u_f32, size):  # noqa: F811
    """Thin matrices whose gram is summed in several parts, some of them zero: the
    zeros say nothing about the size of the others, however small these are.
    eps = 0, and an eps of a millionth of the matrix's size."""
    rng = np.random.default_rng(31)
    zeros = [((100, 1000), slice(256, 384)), ((100, 1000), slice(0, 128)), ((100, 1000), slice(128, 1000)),
             ((60, 700), slice(500, 700)), ((20, 5000), slice(0, 4900)), ((1, 900), slice(100, 900))]
    us = []
    for shape, cols in zeros:
        u = rng.standard_normal(shape) * size
        u[:, cols] = 0.0
        us += [u, u.T.copy()]
    t = Steps(env, us, u_f32)
    for eps in (0.0, 1e-6 * size):
        for got, u in zip(t.o(5, eps=eps), t.u):
            exact = ref.iterate64(u, 5, eps=eps)
            off = np.linalg.norm(got - exact)
            assert off <= 5e-4 * np.linalg.norm(exact), (u.shape, size, eps, off)
    # nothing but zeros in every part
    for got in Steps(env, [np.zeros((100, 1000)), np.zeros((1000, 20))], u_f32).o(5, eps=1e-6 * size):
        assert (got == 0.0).all()
