"""What the number formats alone cost: the iteration with the library's roundings
(and exact products) stays within the figures that the header states, on spectra of
every kind, and is the iteration itself where nothing is rounded away."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest

from tests import muon_formats as fmt
from tests import muon_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("kind", fmt.KINDS)
def test_roundings_stay_within_the_stated_figures(kind):
    rng = np.random.default_rng(3)
    for shape in ((129, 129), (130, 300), (300, 150)):
        u = fmt.spectrum(rng, shape, kind).astype(np.float32)
        for held in (u, ref.widen(ref.bf16(u)).reshape(shape)):
            for steps in (1, 2, 5, 8):
                exact = ref.iterate64(held, steps)
                off = np.linalg.norm(fmt.dense(held, steps) - exact) / np.linalg.norm(exact)
                assert off <= fmt.stated(shape, steps), (shape, steps, off)
                if steps <= 2:
                    # one or two steps hardly amplify anything: roundings of A and B, 2^-11 at most
                    assert off <= 2.0 ** -10, (shape, steps, off)


def test_header_states_these_figures():
    src = open(os.path.join(ROOT, "include", "zero1.h")).read()
    text = re.sub(r"\s*\n \* ?", " ", src)
    for share, steps, shape in (("0.15 %", 5, (128, 300)), ("0.25 %", 8, (128, 300)), ("0.4 %", 5, (129, 300)),
                                ("1.3 %", 8, (129, 300))):
        assert float(share.split()[0]) / 100 == pytest.approx(fmt.stated(shape, steps)), (share, steps)
        assert share in text, share
