"""The exact checks of the router's operators tell right from wrong (CPU): evaluations in the documented
precision pass, and the same with fewer bf16 terms, or fewer bits in a sum, do not."""
import numpy as np
import pytest

import router_exact as X
from test_gpu_router_exact import BACKWARD, DX


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
