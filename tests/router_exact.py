"""Inputs of the balance loss and the router's backward pass on which fp32 arithmetic makes no error,
or hardly any, whatever the order of its sums, and the values that must come out (NumPy only).

Sums of integers, or of multiples of one power of two, are exact in fp32 as long as they stay below
2^24 of it, in every order; a product of bf16 numbers is exact, and so is a sum with nothing but
zeros beside one term.  So a kernel that sums in fp32 gives the value itself, and one that keeps
fewer bits anywhere does not."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def bf16(a):
    """fp32 values rounded to bf16, ties to even."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16
    return u.astype(np.uint32).view(np.float32)


def split(v, terms):
    """v in that many bf16 terms, each the rounding of what the ones before it left; their sum."""
    rest, out = np.asarray(v, np.float32), np.zeros(np.shape(v))
    for _ in range(terms):
        t = bf16(rest)
        out = out + t
        rest = (rest - t).astype(np.float32)
    return out


# ---------------------------------------------------------------- dW_r, db: dl alone
def selection(T, d, E, seed):
    """dl [T, E] with all 24 bits of fp32 and x [T, d] with one 1, -1, 2 or -0.5 a column, in distinct
    rows where T allows it: dw[e, c] = dl[t, e] x[t, c] of the one t, exact.  Where T is below d rows
    repeat, in columns of their own."""
    rng = np.random.default_rng(seed)
    dl = rng.standard_normal((T, E)).astype(np.float32)
    rows = np.concatenate([rng.permutation(T) for _ in range(-(-d // T))])[:d]
    x = np.zeros((T, d), np.float32)
    x[rows, np.arange(d)] = rng.choice([1.0, -1.0, 2.0, -0.5], d)
    dw = dl[rows].astype(np.float64).T * x[rows, np.arange(d)]
    return dl, x, dw


def integers(T, d, E, seed, limit=1 << 24):
    """Integer dl and x whose sums over the tokens stay below 2^24: dw = dl^T x and db = sum dl are
    exact in fp32 in any order.  dl needs two bf16 terms (up to 2^10 where T allows it)."""
    rng = np.random.default_rng(seed)
    top = max(1, min(1023, (limit - 1) // (2 * T)))
    dl = rng.integers(-top, top + 1, (T, E)).astype(np.float32)
    x = rng.integers(-2, 3, (T, d)).astype(np.float32)
    return dl, x, dl.astype(np.float64).T @ x, dl.sum(axis=0, dtype=np.float64)


def dx_integers(T, d, E, seed):
    """dl integers of 15 bits (two bf16 terms), W_r of 0, 1 and -1 with at most 255 terms a sum, and an
    addend that takes the leading bits of dl W_r away: the sums are integers below 2^24, exact in
    fp32, and dx, their rounding, shows dl's last bits."""
    rng = np.random.default_rng(seed)
    dl = rng.integers(-(1 << 15) + 1, 1 << 15, (T, E)).astype(np.float32)
    w = rng.integers(-1, 2, (E, d)).astype(np.float32)
    sums = dl.astype(np.float64) @ w
    add = -bf16(sums.astype(np.float32))
    return dl, w, add, sums + add


# ---------------------------------------------------------------- balance loss
def balance_subsets(T, E, k, seed, masked):
    """Rows with one value (any, e.g. 3.25) on 2^j experts and -inf on the rest: probabilities 2^-j
    or 0, exact, and so their sums over tokens and their products with counts (multiples of 1/256
    below 2^16 of them).  ids: the row's first k experts of a random order, any of the E."""
    rng = np.random.default_rng(seed)
    order = np.argsort(rng.random((T, E)), axis=1)
    most = int(np.log2(E))
    j = rng.integers(0, most + 1, T)
    p = np.zeros((T, E))
    for t in range(T):
        p[t, order[t, :1 << j[t]]] = 0.5 ** j[t]
    value = rng.integers(-40, 41, (T, 1)) / 4.0
    logits = np.where(p > 0, value, -np.inf).astype(np.float32)
    # experts of a skewed preference, so that the counts differ
    score = rng.random((T, E)) + np.linspace(0, 1.5, E)
    ids = np.argsort(-score, axis=1)[:, :k].astype(np.int32)
    mask = (rng.random(T) < 0.8).astype(np.uint8) if masked else None
    return logits, ids, mask, p


def balance_values(p, ids, mask, coef, grad_scale):
    """loss, counts, probs, dlogits of probabilities p, in 64 bits."""
    T, E = p.shape
    k = ids.shape[1]
    keep = np.ones(T, bool) if mask is None else mask != 0
    n = int(keep.sum())
    c = np.bincount(ids[keep].ravel(), minlength=E)
    grad = np.zeros((T, E))
    if n == 0:
        return 0.0, c, np.zeros(E), grad
    above = (c - c.min()).astype(np.float64)
    norm = coef * E / (float(n) * k) / n
    pk = p[keep]
    grad[keep] = grad_scale * norm * pk * (above - (pk @ above)[:, None])
    return norm * float(c @ pk.sum(0)), c, pk.sum(0) / n, grad


# |error| of what comes out, relative: the loss and the mean probabilities are evaluated in 64 bits
# from exact sums and rounded to fp32 once (U, and a little for the evaluation); the gradient's
# factor is rounded to fp32, its two products are (3 U)
LOSS_REL, PROBS_REL, GRAD_REL = 1.001 * U, 1.001 * U, 3.001 * U


def balance_faults(p, ids, mask, coef, grad_scale, got):
    """Names of the outputs that are off by more than the bounds."""
    loss, c, probs, grad = balance_values(p, ids, mask, coef, grad_scale)
    bad = []
    if not np.array_equal(got["counts"], c):
        bad.append("counts")
    if not abs(got["loss"] - loss) <= LOSS_REL * abs(loss):
        bad.append("loss")
    if not np.all(np.abs(got["probs"] - probs) <= PROBS_REL * probs):
        bad.append("probs")
    if not np.all(np.abs(got["dlogits"] - grad) <= GRAD_REL * np.abs(grad)):
        bad.append("dlogits")
    return bad


# ---------------------------------------------------------------- slope of the loss
def directional_faults(x, w, ids, counts, grad_w, coef):
    """Whether grad_w [E, d] is the gradient of the balance loss in W_r, the choices and counts held:
    its slope along D = grad / |grad| of the analytic gradient against the central difference of the
    loss, both in 64 bits.  Returns the difference, its bound and the slope.

    The loss is the mean over tokens of E_p[a] with a_e = coef E c_e / (n k) and p the softmax of z =
    x W^T.  Along D z moves by u_t = x_t D^T.  The third derivative of E_p[a] is the joint cumulant
    of (a, u, u, u): E[a u u u] - 3 E[a u] E[u u] of the centred values, at most 4 A R_t^3 with A
    and R_t the ranges of a and u_t over the experts; the difference is off by h^2 / 6 of its mean,
    and by the loss's rounding, (E + 20) 2^-53 |loss| at either end, over h.  The gradient in fp32: a
    relative 2^-16 of the slope's terms is 256 half steps, far above the (E + 60) U that the softmax,
    the gradient's products and the fp32 sums over some hundred tokens come to."""
    T, E = x.shape[0], w.shape[0]
    k = ids.shape[1]
    a = coef * E * counts / (float(T) * k)

    def loss(wt):
        z = x @ wt.T
        p = np.exp(z - z.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        return float((p @ a).mean()), p

    value, p = loss(w)
    dl = p * (a - (p @ a)[:, None]) / T
    D = dl.T @ x
    D /= np.linalg.norm(D)
    h = 2.0 ** -11
    diff = (loss(w + h * D)[0] - loss(w - h * D)[0]) / (2 * h)
    slope = float((grad_w * D).sum())
    u = x @ D.T
    R = u.max(axis=1) - u.min(axis=1)
    bound = h * h / 6 * float((4 * (a.max() - a.min()) * R ** 3).mean())
    bound += (E + 20) * 2.0 ** -53 * abs(value) / h
    bound += 2.0 ** -16 * float((np.abs(dl).T @ np.abs(x) * np.abs(D)).sum())
    return abs(diff - slope), bound, slope
