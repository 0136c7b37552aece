"""Plain fp64 references of routing by scores, its backward pass and the bias update, and of the
AdamW step (whose moments are fp32 numbers by definition: each operation rounded)."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


# ---------------------------------------------------------------- routing by scores
def scores(z, score):
    """fp64 scores [T, E] of logits [T, E]."""
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        m = z.max(1, keepdims=True)
        m[m == -np.inf] = 0.0
        p = np.exp(z - m)
        total = p.sum(1, keepdims=True)
        total[total == 0.0] = 1.0
        return p / total


def route(z, k, score="softmax", n_groups=1, topk_groups=1, group_score="max", renormalize=False,
          scale=1.0, score_bias=None, token_mask=None):
    """ids [T, k] and fp64 gates [T, k] of logits z [T, E], one token at a time."""
    T, E = z.shape
    s = scores(z.copy(), score)
    ids = np.full((T, k), -1, np.int32)
    gates = np.zeros((T, k))
    bias = np.zeros(E, np.float32) if score_bias is None else score_bias.astype(np.float32)
    on = bias != -np.inf
    order = lambda v: np.inf if np.isnan(v) else v  # NaN above every number
    gs = E // n_groups
    for t in range(T):
        if token_mask is not None and not token_mask[t]:
            continue
        with np.errstate(all="ignore"):
            a = s[t].astype(np.float32) + bias
        rank = lambda e: (not np.isnan(a[e]), -order(a[e]), e)
        allowed = [e for e in range(E) if on[e]]
        if topk_groups < n_groups:
            def strength(g):
                best = sorted((e for e in range(g * gs, (g + 1) * gs) if on[e]), key=rank)
                if not best:
                    return (2, 0.0, g)
                v = a[best[0]]
                if group_score == "top2" and len(best) > 1:
                    with np.errstate(all="ignore"):
                        v = np.float32(v + a[best[1]])
                return (0 if np.isnan(v) else 1, -order(v), g)
            stay = set(sorted(range(n_groups), key=strength)[:topk_groups])
            allowed = [e for e in allowed if e // gs in stay]
        chosen = sorted(allowed, key=rank)[:k]
        if not chosen:
            continue
        ids[t, :len(chosen)] = chosen
        v = s[t, chosen]
        if renormalize:
            zc = z[t, chosen]
            with np.errstate(all="ignore"):
                if np.isnan(v).any():
                    v = np.full(len(v), np.nan)
                elif zc.max() == -np.inf:
                    v = np.zeros(len(v))
                elif score == "softmax":  # the ratios of e^l
                    v = np.exp(zc - zc.max())
                    v = v / v.sum()
                else:  # e^(l - M) / (1 + e^l), M <= 0
                    M = min(zc.max(), 0.0)
                    v = np.where(zc > 0, 1.0 / (1.0 + np.exp(-zc)), np.exp(np.minimum(zc, 0) - M) /
                                 (1.0 + np.exp(np.minimum(zc, 0))))
                    v = v / v.sum()
        gates[t, :len(chosen)] = scale * v
    return ids, gates


def gates_of(z, ids, score, renormalize, scale):
    """fp64 gates of given ids (those outside [0, E) have 0), as a function of the logits."""
    T, E = z.shape
    s = scores(z.copy(), score)
    real = (ids >= 0) & (ids < E)
    v = np.where(real, np.take_along_axis(s, np.where(real, ids, 0).astype(np.int64), 1), 0.0)
    if renormalize:
        total = v.sum(1, keepdims=True)
        v = v / np.where(total == 0.0, 1.0, total)
    return scale * v


def route_backward(z, ids, dgates, score, renormalize, scale, add=None, token_mask=None):
    """dlogits [T, E] in fp64 and a bound on the fp32 kernel's error.  The bound counts roundings: an
    exponential is within 4 of them, a sum of n terms within n, products and quotients one each; at
    most E + k + 40 in all of any term, of the size of the terms."""
    T, E = z.shape
    k = ids.shape[1]
    dl, size = np.zeros((T, E)), np.zeros((T, E))
    s = scores(z.copy(), score)
    for t in range(T):
        if token_mask is not None and not token_mask[t]:
            continue
        cs = [c for c in range(k) if 0 <= ids[t, c] < E]
        e = ids[t, cs].astype(int)
        dg = scale * dgates[t, cs]
        if renormalize:
            zc = z[t, e]
            if len(cs) and zc.max() > -np.inf:
                if score == "softmax":
                    w = np.exp(zc - zc.max())
                else:
                    M = min(zc.max(), 0.0)
                    w = np.where(zc > 0, 1 / (1 + np.exp(-np.maximum(zc, 0))),
                                 np.exp(np.minimum(zc, 0) - M) / (1 + np.exp(np.minimum(zc, 0))))
                q = w / w.sum()
                h = q * (dg - (q * dg).sum())
                b = q * (np.abs(dg) + (q * np.abs(dg)).sum())
                if score == "sigmoid":
                    rest = 1.0 / (1.0 + np.exp(zc))
                    h, b = h * rest, b * rest
                np.add.at(dl[t], e, h)
                np.add.at(size[t], e, b)
        else:
            u, au = np.zeros(E), np.zeros(E)
            np.add.at(u, e, dg)
            np.add.at(au, e, np.abs(dg))
            if score == "sigmoid":
                rest = 1.0 / (1.0 + np.exp(z[t]))
                dl[t] = u * s[t] * rest
                size[t] = au * s[t] * rest
            else:
                dl[t] = s[t] * (u - (s[t] * u).sum())
                size[t] = s[t] * (au + (s[t] * au).sum())
        if add is not None:
            dl[t] += add[t]
            size[t] += np.abs(add[t])
    return dl, (E + k + 40) * U * size + 2.0 ** -140  # what a denormal loses


def balance_bias(ids, E, rate, bias, token_mask=None):
    """The updated bias (fp32) and the counts."""
    keep = ids if token_mask is None else ids[token_mask > 0]
    keep = keep[(keep >= 0) & (keep < E)]
    counts = np.bincount(keep.ravel(), minlength=E)
    on = bias != -np.inf
    total, n = int(counts[on].sum()), int(on.sum())
    out = bias.astype(np.float32).copy()
    for e in range(E):
        if on[e]:
            d = total - n * int(counts[e])
            out[e] = np.float32(out[e] + np.float32(rate) * np.float32((d > 0) - (d < 0)))
    return out, counts


# ---------------------------------------------------------------- AdamW
F = np.float32


def encode(x, top):
    """Codes and steps of fp32 x in blocks of 256 (the last may be short)."""
    n = len(x)
    nb = -(-n // 256)
    v = np.zeros(nb * 256, F)
    v[:n] = x
    v = v.reshape(nb, 256)
    with np.errstate(all="ignore"):
        step = (np.abs(v).max(1) / F(top * top)).astype(F)
        y = np.where(step[:, None] > 0, np.abs(v) / step[:, None], F(0)).astype(F)
        c = np.floor(np.sqrt(y) + F(0.5))
    c = np.where(c >= 0, np.minimum(c, F(top)), F(0)).astype(np.int32)
    if top == 255:
        c = np.where((v > 0) & (c < 1), 1, c)
    else:
        c = np.where(v < 0, -c, c)
    return c.reshape(-1)[:n].astype(np.uint8 if top == 255 else np.int8), step


def decode(code, step):
    c = code.astype(np.int32)
    s = np.repeat(step, 256)[:len(c)]
    with np.errstate(all="ignore"):
        return ((c * np.abs(c)).astype(F) * s).astype(F)


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, wd, grad_scale=1.0):
    """fp64 params, their bound, and the fp32 moments (bits) of one step from fp32 m and v."""
    b1, b2 = F(beta1), F(beta2)
    with np.errstate(all="ignore"):
        g = (g.astype(F) * F(grad_scale)).astype(F)
        m = (m * b1 + g * (F(1) - b1)).astype(F)
        v = (v * b2 + (g * g) * (F(1) - b2)).astype(F)
        lr, wd, eps = float(F(lr)), float(F(wd)), float(F(eps))
        c1 = -np.expm1(step * np.log(float(b1))) if b1 > 0 else 1.0
        c2 = -np.expm1(step * np.log(float(b2))) if b2 > 0 else 1.0
        up = lr * (m.astype(np.float64) / c1) / (np.sqrt(v.astype(np.float64) / c2) + eps)
        p64 = p.astype(np.float64)
        new = p64 - lr * wd * p64 - up
        # update: in half steps of fp32, the factor 1, its product with m 1, the root 1 (2 at 8 bits, the
        # hardware's own), its factor 1, their sum 1, the quotient 1 (2 at 8 bits: reciprocal), so at
        # most 8, and 9 with the second order; p: lr wd, the decayed p, the difference
        bound = U * (9 * np.abs(up) + (1 + lr * wd) * np.abs(p64) + np.abs(new)) + 2.0 ** -140
    return new, bound, m, v
