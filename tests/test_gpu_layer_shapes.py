"""Long batches of the operators that do not look at the token rows, through layer.py."""
from __future__ import annotations

import pytest
import torch

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


def test_gradients_and_bias_of_long_batches():
    """2^26 tokens and a few: one block of tokens repeated gives the same bits everywhere."""
    Tb, T, E = 4096, (1 << 26) + 4096, 2
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of free device memory")
    g = torch.Generator(device=DEV).manual_seed(2)
    reps = T // Tb
    logits, dg = torch.randn(Tb, E, generator=g, device=DEV), torch.randn(Tb, 1, generator=g, device=DEV)
    ids = torch.randint(0, E, (Tb, 1), generator=g, device=DEV, dtype=torch.int32)
    long = lambda t: t.repeat(reps, 1)
    routing = B.make_routing("sigmoid")
    dl = L.route_scored_backward(long(logits), long(ids), long(dg), routing).view(reps, Tb, E)
    want = L.route_scored_backward(logits, ids, dg, routing)
    assert bool((dl == want).all())
    bias = torch.zeros(E, device=DEV)
    counts = L.balance_bias(long(ids), bias, 0.5)
    once = torch.bincount(ids.flatten(), minlength=E)
    assert torch.equal(counts.long(), once * reps)
    assert torch.equal(bias, 0.5 * torch.sign(once.sum() - 2 * once).float())
