"""Plain 64-bit references of the balance loss and of the router's backward pass, and bounds on
what fp32 evaluation may add to them.  NumPy only."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32
# Below 2^-126 fp32 has no full-precision values and the hardware's 2^x gives none at all: every
# probability is off by up to 2^-126 on top of its relative error, whatever its size.  The shift
# carries over to what is linear in the probabilities.
TINY = 2.0 ** -126
BF = 2.0 ** -8  # half a step of bf16, relative (torch.finfo(torch.bfloat16).eps / 2)


def softmax(logits):
    z = np.asarray(logits, np.float64)
    m = z.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.exp(z - m)
        p = p / p.sum(axis=1, keepdims=True)
    p[np.isneginf(m[:, 0])] = 0.0
    return p


def counts_of(ids, E, keep):
    c = np.zeros(E, np.int64)
    for t in np.nonzero(keep)[0]:
        for e in ids[t]:
            if 0 <= e < E:
                c[e] += 1
    return c


def balance(logits, ids, mask=None, coef=1.0, grad_scale=1.0, counts=None):
    """loss, counts, probs, dlogits; `counts` overrides the counts (constants of the gradient)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k = ids.shape[1]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    n = int(keep.sum())
    c = counts_of(ids, E, keep) if counts is None else counts
    grad = np.zeros((T, E))
    if n == 0:
        return 0.0, c, np.zeros(E), grad
    p = softmax(logits[keep])
    S = p.sum(axis=0)
    norm = coef * E / (float(n) * k) / n
    above = (c - c.min()).astype(np.float64)
    grad[keep] = grad_scale * norm * p * (above[None, :] - (p @ above)[:, None])
    return norm * float(c @ S), c, S / n, grad


def softmax_bound(logits, E):
    """Relative error of one fp32 probability: the subtraction (|l - max| u, as exp turns it into
    a relative one), exp (2 steps), the sum of E terms, the reciprocal and the product.  A logit
    120 or more below the row's largest counts for none of it: e^-120 < 2^-149, so fp32 has 0 there
    and the bounds' terms in TINY cover the probability."""
    z = np.where(np.isfinite(logits), np.asarray(logits, np.float64), 0.0)
    if not len(z):
        return np.zeros((0, 1))
    m = z.max(axis=1, keepdims=True)
    spread = m - np.where(z >= m - 120, z, m).min(axis=1, keepdims=True)
    return (2 * spread + E + 12) * U


def balance_bounds(logits, ids, mask, coef, grad_scale):
    """Bounds on |error| of loss, probs and dlogits (all sums have terms of one sign but the
    gradient's, which is bounded against the largest count difference)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    loss, c, probs, grad = balance(logits, ids, mask, coef, grad_scale)
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    n = max(int(keep.sum()), 1)
    # a lane adds at most T / 8 + 1 tokens one after another (one block of 8 waves), then lanes
    # and waves; capped at 1024 blocks' worth of tokens a lane
    adds = min(T // 8 + 1, T // 256 + 1024) + 80
    rp = softmax_bound(np.where(keep[:, None], logits, 0.0), E)
    rel = (rp.max() if T else 0.0) + adds * U + 4 * U
    p = np.zeros((T, E))
    p[keep] = softmax(logits[keep])
    norm = abs(grad_scale) * coef * E / (float(n) * ids.shape[1]) / n
    above = float((c - c.min()).max())
    g = norm * above * (p * (3 * rp + (2 * E + 8) * U) + (E + 1) * TINY)
    # (c_e / (n k) sums to at most 1; the last TINY is the result's own)
    return rel * abs(loss) + (abs(coef) * E + 1) * TINY, rel * probs + 2 * TINY, g + TINY


def route_backward(x, w, logits, ids, dgates, dlogits, mask=None, add=None):
    """dx, dw, db and dl (the gradient on the logits)."""
    T, d = x.shape
    E = w.shape[0]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    dl = np.zeros((T, E))
    if dgates is not None:
        dp = np.zeros((T, E))
        for t in np.nonzero(keep)[0]:
            for c in range(ids.shape[1]):
                if 0 <= ids[t, c] < E:
                    dp[t, ids[t, c]] += float(dgates[t, c])
        p = np.zeros((T, E))
        p[keep] = softmax(logits[keep])
        dl = p * (dp - (p * dp).sum(axis=1, keepdims=True))
    if dlogits is not None:
        dl[keep] += np.asarray(dlogits, np.float64)[keep]
    x64 = np.where(keep[:, None], np.asarray(x, np.float64), 0.0)
    dx = dl @ np.asarray(w, np.float64)
    if add is not None:
        dx = dx + np.asarray(add, np.float64)
    return dx, dl.T @ x64, dl.sum(axis=0), dl


def route_backward_bounds(x, w, logits, ids, dgates, dlogits, mask, add, bf16):
    """Bounds on |error| of dx, dw, db, element by element."""
    T, d = x.shape
    E, k = w.shape[0], ids.shape[1] if ids is not None else 0
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    dx, dw, db, dl = route_backward(x, w, logits, ids, dgates, dlogits, mask, add)
    ddl = 3 * U * np.abs(dl)
    if dgates is not None:
        p, dp = np.zeros((T, E)), np.zeros((T, E))
        p[keep] = softmax(logits[keep])
        for t in np.nonzero(keep)[0]:
            for c in range(k):
                if 0 <= ids[t, c] < E:
                    dp[t, ids[t, c]] += abs(float(dgates[t, c]))
        rp = softmax_bound(np.where(keep[:, None], logits, 0.0), E)
        ddl += p * (dp + (p * dp).sum(axis=1, keepdims=True)) * (3 * rp + (E + k + 8) * U)
        ddl += (E + 2) * dp.sum(axis=1, keepdims=True) * TINY
    if dlogits is not None:
        ddl[keep] += 2 * U * np.abs(np.asarray(dlogits, np.float64)[keep])
    aw = np.abs(np.asarray(w, np.float64))
    ax = np.where(keep[:, None], np.abs(np.asarray(x, np.float64)), 0.0)
    adl = np.abs(dl) + ddl
    # dx: dl in two bf16 terms (each keeps half a step of what is left: 2^-8 2^-8 in all) in bf16,
    # E products summed in fp32 (twice as many with two terms), the addition, the rounding
    terms = 2 if bf16 else 1
    mag = adl @ aw
    bx = ddl @ aw + mag * ((BF * BF if bf16 else 0.0) + (terms * max(E, 32) + 4) * U)
    bx += (np.abs(dx) + bx) * (BF if bf16 else U)
    if add is not None:
        bx += 2 * U * np.abs(np.asarray(add, np.float64))
    # dw: three terms keep 24 bits and more; every product may be added one after another
    n = (3 if bf16 else 1) * T + 600
    bw = ddl.T @ ax + (adl.T @ ax) * (n + 4) * U
    bb = ddl.sum(axis=0) + adl.sum(axis=0) * (T + 600) * U
    return bx + 1e-40, bw + 1e-40, bb + 1e-40
