"""8-bit moments over many steps, codes to the code: gradients that end, in a block where others go on."""
from __future__ import annotations

import pytest
import torch

from capacity_routing_expert_amd import binding as B
from test_gpu_adamw import DEV, HYPER, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[256], [1000, 257]])
def test_gradients_that_end(lengths):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    c = Case(lengths, 8, seed=12, fresh=True)
    gen = torch.Generator(device=DEV).manual_seed(3)
    for step in range(1, 41):
        for g in c.g:
            g.copy_(torch.randn(g.numel(), generator=gen, device=DEV))
            g[::3] *= 0.01 if step <= 10 else 0.0
        want = c.expect(step)
        B.moe_adamw_step(c.tensors, step=step, **HYPER)
        c.check(want)
    assert all(bool((m[::3] != 0).any()) for m in c.m)  # small codes stay
