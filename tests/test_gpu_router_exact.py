"""moe_balance_loss and moe_route_backward on inputs where fp32 sums make no error (router_exact): the
outputs are the values themselves or their one rounding, for every kernel and length; and the balance
loss's gradient in W_r, end to end, against the difference of the loss along it."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

import router_exact as X
from capacity_routing_expert_amd import binding as B
from capacity_routing_expert_amd import layer as L

pytestmark = pytest.mark.gpu

DEV = "cuda:0"

BACKWARD = [(1, 64, 1), (2, 128, 8), (3, 8, 3), (33, 72, 16), (130, 520, 17), (257, 136, 40),
            (500, 1032, 64), (1000, 72, 130), (700, 64, 256), (5000, 256, 8), (2500, 1032, 4),
            (9000, 2048, 40), (20000, 2048, 64), (33000, 128, 12)]
DX = [(1, 64, 1), (2, 128, 8), (33, 72, 16), (130, 520, 17), (257, 136, 40), (500, 1032, 64),
      (300, 72, 130), (200, 64, 250), (5000, 256, 8), (9000, 1032, 5)]
BALANCE = [(1, 1, 1), (1, 2, 1), (5, 3, 2), (64, 8, 2), (700, 12, 3), (1023, 16, 1), (515, 32, 6),
           (4097, 64, 6), (1000, 65, 4), (2049, 100, 8), (777, 130, 8), (3000, 256, 8), (9000, 8, 2),
           (20000, 60, 4)]


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    B.lib()  # loud failure if the library is missing
    yield
    torch.cuda.synchronize()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,d,E", BACKWARD)
def test_dw_takes_every_bit_of_dl(T, d, E, bf16):
    """One product a sum: dW_r holds dl's 24 bits, in bf16 through all three terms."""
    say(f"[dw, one product] T={T} d={d} E={E} bf16={bf16}")
    dt = torch.bfloat16 if bf16 else torch.float32
    dl, x, dw = X.selection(T, d, E, T + E)
    got = L.route_backward(dev(x, dt), dev(np.zeros((E, d), np.float32), dt), None, None,
                           dlogits=dev(dl))
    assert np.array_equal(host(got["dw_router"]), dw)
    assert not host(got["dx"]).any()


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,d,E", BACKWARD)
def test_sums_over_tokens_are_exact(T, d, E, bf16, masked):
    """Integers whose sums stay below 2^24: dW_r and db are the integers."""
    say(f"[dw, db, integers] T={T} d={d} E={E} bf16={bf16} masked={masked}")
    dt = torch.bfloat16 if bf16 else torch.float32
    dl, x, dw, db = X.integers(T, d, E, T + E)
    mask = None
    if masked:
        m = np.random.default_rng(T).random(T) < 0.7
        dw, db = dl[m].astype(np.float64).T @ x[m], dl[m].sum(axis=0, dtype=np.float64)
        x[~m], dl[~m] = np.nan, np.inf
        mask = dev(m.astype(np.uint8))
    got = L.route_backward(dev(x, dt), dev(np.zeros((E, d), np.float32), dt), None, None,
                           dlogits=dev(dl), token_mask=mask)
    assert np.array_equal(host(got["dw_router"]), dw)
    assert np.array_equal(host(got["db_router"]), db)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,d,E", DX)
def test_dx_is_one_rounding(T, d, E, bf16):
    """dl of 15 bits (two bf16 terms) times W_r of 0 and +-1, plus an addend: exact sums, so dx is
    their rounding to bf16, or the sum itself in f32."""
    say(f"[dx, integers] T={T} d={d} E={E} bf16={bf16}")
    dt = torch.bfloat16 if bf16 else torch.float32
    dl, w, add, dx = X.dx_integers(T, d, E, T + E)
    got = L.route_backward(dev(np.zeros((T, d), np.float32), dt), dev(w, dt), None, None,
                           dlogits=dev(dl), dx_add=dev(add, dt))
    want = X.bf16(dx.astype(np.float32)).astype(np.float64) if bf16 else dx
    assert np.array_equal(host(got["dx"]), want)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", BALANCE)
def test_balance_of_exact_probabilities(T, E, k, masked):
    say(f"[balance, exact probabilities] T={T} E={E} k={k} masked={masked}")
    logits, ids, mask, p = X.balance_subsets(T, E, k, T + E, masked)
    coef, scale = 0.3125, -1.5
    got = L.balance_loss(dev(logits), dev(ids), coef=coef, grad_scale=scale,
                         token_mask=None if mask is None else dev(mask))
    got = dict(loss=float(got["loss"]), counts=host(got["counts"]), probs=host(got["probs"]),
               dlogits=host(got["dlogits"]))
    assert X.balance_faults(p, ids, mask, coef, scale, got) == []


def slope_case():
    """x, W_r, the choices and coef of a router whose experts are far from evenly used."""
    rng = np.random.default_rng(9)
    T, d, E, k = 256, 64, 8, 2
    x = rng.standard_normal((T, d)).astype(np.float32).astype(np.float64)
    x[:, 0] = 1.0  # a common part, on which the experts' preferences differ
    w = (rng.standard_normal((E, d)) / 8).astype(np.float32)
    w[:, 0] = np.linspace(-1, 1, E).astype(np.float32)
    w = w.astype(np.float64)
    ids = np.argsort(-(x @ w.T), axis=1, kind="stable")[:, :k].astype(np.int32)
    return x, w, ids, 1.0


@pytest.mark.parametrize("bf16", [False, True])
def test_gradient_is_the_slope_of_the_loss(bf16):
    """moe_route, moe_balance_loss and moe_route_backward: the gradient in W_r against the difference
    of the loss along it."""
    x, w, _, coef = slope_case()
    if bf16:
        x, w = (X.bf16(a.astype(np.float32)).astype(np.float64) for a in (x, w))
    (T, d), E, k = x.shape, w.shape[0], 2
    dt = torch.bfloat16 if bf16 else torch.float32
    xd, wd = dev(x, dt), dev(w, dt)
    shape = B.make_shape(T, d, 8, E, k, 0, B.MOE_BF16 if bf16 else B.MOE_F32)
    ws = torch.empty(max(B.workspace_bytes(shape), 256), dtype=torch.uint8, device=DEV)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    gates, logits = torch.empty(T, k, device=DEV), torch.empty(T, E, device=DEV)
    B.moe_route(shape, xd, wd, None, ids, gates, logits, ws)
    bal = L.balance_loss(logits, ids, coef=coef)
    got = L.route_backward(xd, wd, logits, ids, dlogits=bal["dlogits"])
    off, bound, slope = X.directional_faults(x, w, ids.cpu().numpy(), host(bal["counts"]),
                                             host(got["dw_router"]), coef)
    say(f"[slope] off {off:.2e} bound {bound:.2e} slope {slope:.4f}")
    assert off <= bound
