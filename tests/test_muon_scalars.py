"""The Muon scalars of a captured step, derived from the same hyper-parameters that
the captured calls are given (no GPU)."""
from __future__ import annotations

import zero_sharded_mixed_zero1_amd as z


def test_derive_reads_the_values_beside_device_scalars():
    """As in C, the device address is ignored; the values are what is derived."""
    hp = dict(lr=3e-4, momentum=0.95, weight_decay=0.1, max_norm=0.5)
    want = bytes(z.muon_scalars_derive(hp))
    assert bytes(z.muon_scalars_derive(dict(hp, device_scalars=1 << 40))) == want
    h = z.MuonHParams(3e-4, 0.95, 0.1, 0.5, 0.0, 0.0, 0.0, 0.0, 0, 0, 1 << 40)
    assert bytes(z.muon_scalars_derive(h)) == want
