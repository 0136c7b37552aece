"""Shapes that layer.py makes for operators which do not look at the token rows: no limit of the rows'
size is theirs (no GPU: tensors without storage, calls recorded)."""
import pytest
import torch

from capacity_routing_expert_amd import binding as B
from capacity_routing_expert_amd import layer as L


@pytest.mark.parametrize("T", [1, (1 << 26) - 1, 1 << 26, (1 << 29) - 1])
@pytest.mark.parametrize("call", ["backward", "bias"])
def test_long_batches(monkeypatch, T, call):
    """Up to 2^29 tokens, where x of one fp32 column would reach 2 GiB."""
    shapes = []
    for name in ("moe_route_scored_backward", "moe_balance_bias"):
        monkeypatch.setattr(B, name, lambda shape, *a, **kw: shapes.append(shape))
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="meta")
    logits, ids = e(T, 4), e(T, 2, dt=torch.int32)
    if call == "backward":
        L.route_scored_backward(logits, ids, e(T, 2), B.make_routing())
    else:
        L.balance_bias(ids, e(4), 0.01)
    assert shapes[0].T == T
    assert B.workspace_bytes(shapes[0]) > 0, B.last_error()
