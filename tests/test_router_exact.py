"""The exact checks of the router's operators tell right from wrong (CPU): evaluations in the documented
precision pass, and the same with fewer bf16 terms, fewer bits in a sum or a wrong gradient do not."""
import numpy as np
import pytest

import router_exact as X
from test_gpu_router_exact import BALANCE, BACKWARD, DX, slope_case


@pytest.mark.parametrize("T,d,E", BACKWARD)
def test_three_terms_give_dw_and_fewer_do_not(T, d, E):
    dl, x, dw = X.selection(T, d, E, T + E)
    rows = np.abs(x).argmax(axis=0)
    at = x[rows, np.arange(d)].astype(np.float64)
    for terms, right in ((3, True), (2, False), (1, False)):
        assert np.array_equal(X.split(dl, terms)[rows].T * at, dw) == right, terms
    dl, x, dw, db = X.integers(T, d, E, T + E)
    assert np.abs(dw).max() < 1 << 24 and np.abs(db).max() < 1 << 24
    assert (np.abs(dl).T @ np.abs(x)).max() < 1 << 24 and np.abs(dl).sum(0).max() < 1 << 24
    assert np.array_equal(X.split(dl, 2), dl)
    if T >= 64:  # a sum that is rounded to bf16 on its way
        half = X.bf16((dl[: T // 2].T @ x[: T // 2]).astype(np.float32)).astype(np.float64)
        assert not np.array_equal(half + dl[T // 2:].T.astype(np.float64) @ x[T // 2:], dw)


@pytest.mark.parametrize("T,d,E", DX)
def test_two_terms_give_dx_and_one_does_not(T, d, E):
    dl, w, add, dx = X.dx_integers(T, d, E, T + E)
    assert (np.abs(dl) @ np.abs(w) + np.abs(add)).max() < 1 << 24
    for terms, right in ((2, True), (1, False)):
        got = X.bf16((X.split(dl, terms) @ w + add).astype(np.float32))
        assert np.array_equal(got, X.bf16(dx.astype(np.float32))) == right, terms


@pytest.mark.parametrize("T,E,k", BALANCE)
def test_balance_values_tell_fewer_bits(T, E, k):
    logits, ids, mask, p = X.balance_subsets(T, E, k, T + E, True)
    if not mask.any():
        mask[0] = 1
    coef, scale = 0.3125, -1.5
    loss, c, probs, grad = X.balance_values(p, ids, mask, coef, scale)
    f32 = lambda a: np.asarray(a, np.float32).astype(np.float64)
    right = dict(loss=float(f32(loss)), counts=c, probs=f32(probs), dlogits=f32(grad))
    assert X.balance_faults(p, ids, mask, coef, scale, right) == []
    less = lambda a: X.bf16(f32(a).astype(np.float32)).astype(np.float64).reshape(np.shape(a))
    step = lambda a: f32(a) * (1 + 4 * X.U)  # two whole steps of fp32
    for wrong in (less, step):
        for name in ("loss", "probs", "dlogits"):
            bad = dict(right, **{name: wrong(right[name])})
            same = np.array_equal(bad[name], right[name])  # zeros, or few bits to begin with
            assert X.balance_faults(p, ids, mask, coef, scale, bad) == ([] if same else [name])
            assert not same or wrong is less or not np.any(right[name])
    bad = dict(right, counts=c + (np.arange(E) == 0))
    assert X.balance_faults(p, ids, mask, coef, scale, bad) == ["counts"]


def test_the_slope_tells_a_wrong_gradient():
    x, w, ids, coef = slope_case()
    T, E = len(x), len(w)
    counts = np.bincount(ids.ravel(), minlength=E).astype(np.float64)
    z = x @ w.T
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    a = coef * E * counts / (float(T) * ids.shape[1])
    dl = p * (a - (p @ a)[:, None]) / T
    right = dl.T @ x
    f32 = right.astype(np.float32).astype(np.float64)
    off, bound, slope = X.directional_faults(x, w, ids, counts, f32, coef)
    assert off <= bound and bound <= 2e-3 * slope, (off, bound, slope)
    no_dot = (p * a / T).T @ x            # without the softmax's coupling
    half = (dl * (np.arange(E) % 2)).T @ x  # half of the experts left out
    for wrong in (-f32, 2 * f32, 1.005 * f32, 0 * f32, no_dot, half, f32[::-1], f32[:, ::-1]):
        off, bound, _ = X.directional_faults(x, w, ids, counts, wrong, coef)
        assert off > bound
