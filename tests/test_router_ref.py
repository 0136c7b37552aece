"""The 64-bit references of the balance loss and the router's backward pass against central
differences (CPU)."""
import numpy as np
import pytest

import router_ref as R


@pytest.mark.parametrize("T,E,k,masked", [(1, 2, 1, False), (5, 4, 2, True), (7, 6, 3, False)])
def test_balance_gradient_is_the_loss_difference(T, E, k, masked):
    rng = np.random.default_rng(T * 10 + E)
    logits = rng.standard_normal((T, E))
    ids = np.argsort(-logits, axis=1)[:, :k]
    mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
    _, c, _, grad = R.balance(logits, ids, mask, coef=0.3)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            a, b = logits.copy(), logits.copy()
            a[t, e] += h
            b[t, e] -= h
            diff = (R.balance(a, ids, mask, 0.3, counts=c)[0] -
                    R.balance(b, ids, mask, 0.3, counts=c)[0]) / (2 * h)
            # central difference: h^2 times a third derivative (at most the loss's size), and
            # the loss's rounding over h
            assert abs(diff - grad[t, e]) <= 1e-9


@pytest.mark.parametrize("T,d,E,k", [(1, 3, 2, 1), (4, 5, 4, 2)])
def test_route_backward_is_the_gates_difference(T, d, E, k):
    """Of sum dgates * gates + sum dlogits * logits as a function of x, W and b, the choices held."""
    rng = np.random.default_rng(T + d)
    x, w, b = rng.standard_normal((T, d)), rng.standard_normal((E, d)), rng.standard_normal(E)
    logits = x @ w.T + b
    ids = np.argsort(-logits, axis=1)[:, :k]
    dg, dlg = rng.standard_normal((T, k)), rng.standard_normal((T, E))

    def value(x, w, b):
        L = x @ w.T + b
        return (np.take_along_axis(R.softmax(L), ids, 1) * dg).sum() + (L * dlg).sum()

    dx, dw, db, _ = R.route_backward(x, w, logits, ids, dg, dlg)
    h = 1e-5
    for arr, grad in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + h
            hi = value(x, w, b)
            arr[i] = old - h
            lo = value(x, w, b)
            arr[i] = old
            assert abs((hi - lo) / (2 * h) - grad[i]) <= 1e-7
