"""8-bit matrices on the GPU at the edges of what the header allows: products without
rows."""
from __future__ import annotations

import numpy as np
import pytest

import zero_sharded_mixed_zero1_amd as z
from tests.gpu_util import torch_cuda
from tests.test_gpu_f8 import Mat

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, dev


@pytest.mark.parametrize("rows", [7, 64, 300])
@pytest.mark.parametrize("f32", [False, True])
def test_products_without_rows_need_no_workspace(env, rows, f32):
    """A long summed axis, which a product with rows would take in parts, and one operand without rows: nothing is written."""
    torch, dev = env
    k, flags = 8192, z.F32 if f32 else 0
    some = Mat(env, rows, k).put(np.full((rows, k), 0x38, np.uint8), np.full((rows, k // 128), 127, np.uint8))
    none = z.f8_matrix(0, k, None, None)
    d = torch.full((rows, 8), 5.0, device=dev, dtype=torch.float32 if f32 else torch.bfloat16)
    for a, b in ((some.m, none), (none, some.m), (none, none)):
        assert z.f8_product_workspace_bytes(a, b, flags) == 0
        z.f8_product(a, b, d, flags=flags)
        z.f8_product(a, b, None, flags=flags)
    torch.cuda.synchronize()
    assert (d == 5.0).all()
