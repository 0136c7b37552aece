"""The references of routing by scores against small cases worked by hand and against differences."""
import numpy as np
import pytest

import scored_ref as S


def test_choice_by_hand():
    z = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))  # softmax: 1/8, 1/4, 1/2, 1/8
    ids, g = S.route(z, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(g, [[0.5, 0.25]])
    # the bias moves the choice, not the gate
    ids, g = S.route(z, 2, score_bias=np.array([1, 0, 0, 0], np.float32))
    assert ids.tolist() == [[0, 2]] and np.allclose(g, [[0.125, 0.5]])
    ids, g = S.route(z, 2, renormalize=True, scale=3.0)
    assert np.allclose(g, [[2.0, 1.0]])
    # groups {0, 1} and {2, 3}: best single 1/2 against sums 3/8 and 5/8
    ids, _ = S.route(z, 2, n_groups=2, topk_groups=1)
    assert ids.tolist() == [[2, 3]]
    ids, _ = S.route(z, 2, n_groups=2, topk_groups=1, group_score="top2",
                     score_bias=np.array([0.25, 0.125, -0.25, 0], np.float32))
    assert ids.tolist() == [[0, 1]]  # .375 + .375 against .25 + .125, ties to the lower expert
    ids, _ = S.route(z, 4, score_bias=np.array([0, -np.inf, 0, -np.inf], np.float32))
    assert ids.tolist() == [[2, 0, -1, -1]]


def test_scores_out_of_range():
    z = np.array([[-900.0, -901.0, -5000.0], [-np.inf, -np.inf, -np.inf]])
    ids, g = S.route(z, 2, score="sigmoid", renormalize=True)
    assert np.allclose(g[0], np.array([1, np.exp(-1)]) / (1 + np.exp(-1))) and np.all(g[1] == 0)
    assert ids.tolist() == [[0, 1], [0, 1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_backward_against_differences(score, renormalize):
    rng = np.random.default_rng(1)
    T, E, k, scale, h = 6, 7, 3, 2.5, 1e-6
    z = rng.normal(size=(T, E)) * 2
    ids = np.argsort(-z, 1)[:, :k].astype(np.int32)
    ids[1, 2] = -1
    ids[2, 1] = ids[2, 0]  # an expert twice
    dg = rng.normal(size=(T, k))
    dl, _ = S.route_backward(z, ids, dg, score, renormalize, scale)
    loss = lambda y: (S.gates_of(y, ids, score, renormalize, scale) * dg).sum(1)
    for e in range(E):
        d = np.zeros_like(z)
        d[:, e] = h
        assert np.allclose((loss(z + d) - loss(z - d)) / (2 * h), dl[:, e], atol=1e-8)


def test_bias_update_by_hand():
    ids = np.array([[0, 1], [0, 2], [0, -1]], np.int32)
    b, c = S.balance_bias(ids, 4, 0.5, np.array([0, 0, 0, -np.inf], np.float32))
    assert c.tolist() == [3, 1, 1, 0] and b.tolist() == [-0.5, 0.5, 0.5, -np.inf]  # 5 against 3 c


def test_codes_by_hand():
    x = np.zeros(300, np.float32)
    x[0], x[1], x[2], x[3], x[299] = 127 ** 2, -9.0, 0.2, 0.26, 16129 * 4
    c, s = S.encode(x, 127)
    assert s.tolist() == [1.0, 4.0] and c[:4].tolist() == [127, -3, 0, 1] and c[299] == 127
    assert S.decode(c, s)[1] == -9.0
    r = np.array([65025.0, 0.01, 0.0], np.float32)
    c, s = S.encode(r, 255)
    assert c.tolist() == [255, 1, 0]


def test_adamw_first_step_is_lr_times_sign():
    p, g = np.zeros(4, np.float32), np.array([1, -2, 1e-3, 0], np.float32)
    z = np.zeros(4, np.float32)
    new, _, m, v = S.adamw(p, g, z, z, 0.1, 0.9, 0.999, 1e-12, 1, 0.0)
    assert np.allclose(new, -0.1 * np.sign(g), rtol=1e-4)
