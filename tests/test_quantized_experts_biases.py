"""Biases of 4-bit experts (no GPU: refused before anything is quantised)."""
import pytest
import torch

from capacity_routing_expert_amd import layer as L


@pytest.mark.parametrize("which", ["b1", "b2", "both"])
def test_gated_experts_with_biases_are_refused(which):
    """They would be left out of the products without a word."""
    w = lambda *n: torch.zeros(n, dtype=torch.bfloat16)
    b1 = w(2, 96) if which != "b2" else None
    b2 = w(2, 64) if which != "b1" else None
    with pytest.raises(ValueError, match="no biases"):
        L.quantize_experts(w(2, 192, 64), b1, w(2, 64, 96), b2, 32, gated=True)
