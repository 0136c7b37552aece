"""Renormalised gates of scores near and below the end of fp64's range: the ratios of the scores as real
numbers, in a row's every mixture of them, for any scale."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scored_ref as S
from capacity_routing_expert_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


def gates_of(z, k, score, scale, bias=None):
    """ids and gates of one token whose logits are z (they come in through the router's bias)."""
    E, d = len(z), 4
    shape = B.make_shape(1, d, 8, E, k, 0, B.MOE_F32)
    ids = torch.full((1, k), 77, dtype=torch.int32, device=DEV)
    gates = torch.full((1, k), 77.0, device=DEV)
    ws = torch.empty(max(B.workspace_bytes_route_scored(shape), 256), dtype=torch.uint8, device=DEV)
    B.moe_route_scored(shape, B.make_routing(score, renormalize=True, scale=scale), torch.zeros(1, d, device=DEV),
                       torch.zeros(E, d, device=DEV), torch.tensor(z, device=DEV),
                       None if bias is None else torch.tensor(bias, device=DEV), ids, gates, ws=ws)
    return ids.cpu().numpy(), gates.double().cpu().numpy()


def check(z, k, score, scale, bias=None):
    ids, gates = gates_of(z, k, score, scale, bias)
    want, ref = S.route(np.array([z]), k, score=score, renormalize=True, scale=float(np.float32(scale)),
                        score_bias=None if bias is None else np.array(bias, np.float32))
    assert np.array_equal(ids, want)
    # one rounding to fp32, and exponentials of arguments up to 2^10, which fp64 holds to 2^-43 each side
    tol = np.abs(ref) * (S.U + 2.0 ** -40) + 2.0 ** -150
    assert np.all(np.abs(gates - ref) <= tol), (gates, ref)
    return ref


SIGMOID = [[-640.0, -720.0, -INF, -650.0], [-640.0, -INF, -720.0, -700.0], [-610.0, -INF, -INF, -INF],
           [-620.0, -710.0, -660.0, -701.0], [-600.0, -700.5, -699.5, -703.0], [-633.0, -633.0, -634.0, -INF],
           [-460.0, -461.0, -530.0, -563.0], [-459.0, -INF, -545.0, -701.0], [-470.0, -744.0, -746.0, -520.0],
           [-575.0, -663.0, -677.0, -690.0], [-644.0, -645.0, -744.0, -748.0], [-700.0, -701.0, -800.0, -INF],
           [-300.0, -390.0, -403.0, -INF], [0.0, -80.0, -102.0, -INF], [40.0, -700.0, -90.0, 30.0]]


@pytest.mark.parametrize("scale", [1.0, 2.5, 1e-30, 3e38])
@pytest.mark.parametrize("z", SIGMOID)
def test_sigmoid(z, scale):
    check(z, 4, "sigmoid", scale)


def test_zero_scores_have_no_gate():
    """-inf beside a score that fp64 holds: a gate of zero, not a small number."""
    for z in ([-640.0, -INF], [-600.0, -INF], [-645.0, -INF], [-400.0, -INF]):
        ids, gates = gates_of(z, 2, "sigmoid", 3e38)
        assert ids.tolist() == [[0, 1]] and gates[0, 1] == 0.0
        assert gates[0, 0] == float(np.float32(3e38))


@pytest.mark.parametrize("scale", [1.0, 1e-30, 3e38])
@pytest.mark.parametrize("below", [[-644.0, -730.0, -650.0], [-600.0, -735.0, -744.0], [-633.0, -633.0, -634.0],
                                   [-460.0, -461.0, -563.0], [-520.0, -608.0, -622.0], [-744.0, -745.0, -800.0],
                                   [-640.0, -INF, -700.0], [-1000.0, -1088.0, -1101.0]])
def test_softmax_far_below_the_row(below, scale):
    """The row's largest logit belongs to an expert that is off."""
    check([0.0, *below], 3, "softmax", scale, bias=[-INF, 0.0, 0.0, 0.0])
