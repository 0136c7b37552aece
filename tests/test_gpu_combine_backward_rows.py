"""Which rows the backward pass of the combine looks at."""
from __future__ import annotations

import pytest
import torch

import scored_ref as S
from capacity_routing_expert_amd import binding as B
from capacity_routing_expert_amd import layer as L

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_rows_without_capacity(dtype):
    """Capacity 0: no expert rows, so none is looked at, whatever slot_of holds."""
    T, d, E, k = 9, 40, 4, 3
    shape = B.make_shape(T, d, 8, E, k, 0, B.MOE_BF16 if dtype is torch.bfloat16 else B.MOE_F32)
    dout, gates = torch.ones(T, d, dtype=dtype, device=DEV), torch.rand(T, k, device=DEV)
    slots = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    slots[1], slots[2] = -1, 2 ** 31 - 1
    for y in (None, torch.empty(0, d, dtype=dtype, device=DEV)):
        dg = torch.full((T, k), 7.0, device=DEV)
        B.moe_combine_backward(shape, dout, gates, slots, y, dgates=dg)
        assert not bool(dg.any())
    x = torch.randn(T, d, device=DEV).to(dtype)
    g = L.combine_backward(shape, x, gates, torch.full_like(slots, -1), torch.empty(0, d, dtype=dtype, device=DEV),
                           want_rows=True)
    assert not bool(g["dgates"].any()) and g["dy_rows"].numel() == 0
