"""Muon plans and calls beside other work of the program's own streams."""
from __future__ import annotations

import numpy as np
import pytest

import zero_sharded_mixed_zero1_amd as z
from tests.test_gpu_muon import env  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["muon", "mta"])
def test_plan_into_memory_that_the_stream_still_writes(env, kind):  # noqa: F811
    """A table allocated on a side stream may be memory that kernels queued on it
    still write (torch reuses a freed tensor's memory in stream order): the plan's
    copy comes after them."""
    torch, dev = env
    if kind == "muon":
        u, o = (torch.zeros(300, 500, dtype=torch.bfloat16, device=dev) for _ in range(2))
        items, table_bytes, make = [z.matrix(300, 500, u=u, o=o)], z.muon_table_bytes, z.muon_plan
    else:
        param = torch.zeros(90000, dtype=torch.bfloat16, device=dev)
        items = [(90000, 0, param, *(torch.zeros(90000, device=dev) for _ in range(3)))]
        table_bytes, make = z.mta_table_bytes, z.mta_plan
    n = table_bytes(items)
    want = torch.zeros(n, dtype=torch.uint8, device=dev)
    make(items, want)
    torch.cuda.synchronize()
    a = torch.randn(4096, 4096, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            old = torch.zeros(n, dtype=torch.uint8, device=dev)
            at = old.data_ptr()
            side.synchronize()
            for _ in range(20):
                a = (a @ a).clamp_(-1, 1)       # (a while of work before the writes)
            old.fill_(0xEE)
            del old
            table = torch.empty(n, dtype=torch.uint8, device=dev)
            assert table.data_ptr() == at, "the memory was not reused"
            plan = make(items, table)
            side.synchronize()
            assert plan.table == at and np.array_equal(table.cpu().numpy(), want.cpu().numpy())
            del table
