"""8-bit moments over many steps, codes to the code: gradients that end, in a block where others go on."""
from __future__ import annotations

import numpy as np
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


@pytest.mark.parametrize("dynamic", [False, True])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_params_with_fp32_moments(grad, dynamic):
    """Seven half steps of the update, two fewer than the reference's bound, which holds for 8 bits' hardware
    roots and reciprocals too: rate, its product with m, the root, its factor, their sum, the quotient,
    one for the second order."""
    c = Case([100003, 257], 32, grad=grad, seed=13)
    for step in (1, 5):
        before = [c.host(i)[0].astype(np.float64) for i in range(2)]
        want = c.expect(step)
        dyn = torch.tensor([HYPER["lr"], 1.0, step, 0.0], device=DEV) if dynamic else None
        B.moe_adamw_step(c.tensors, step=step, dynamic=dyn, **HYPER)
        c.check(want)
        lr = float(np.float32(HYPER["lr"]))
        for i, (p, bound, _, _) in enumerate(want):
            up = before[i] - lr * float(np.float32(c.wd[i])) * before[i] - p
            got = c.p[i].double().cpu().numpy()
            assert np.all(np.abs(got - p) <= bound - 2 * 2.0 ** -24 * np.abs(up)), i
