"""Plain references of the 4-bit expert weights and of the expert products on them, in 64 bits (the
quantiser in fp32, which defines it).  NumPy only."""
from __future__ import annotations

import numpy as np

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U, BF = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative


def bf16(a):
    """fp32 values rounded to bf16, ties to even."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16
    return u.astype(np.uint32).view(np.float32)


def quantize(w, group):
    """codes [E, rows, cols] (0 .. 15) and scales [E, rows, ceil(cols / group)] fp32 (bf16 values)."""
    w = np.asarray(w, np.float32)
    E, rows, cols = w.shape
    G = -(-cols // group)
    v = np.zeros((E, rows, G * group), np.float32)
    v[:, :, :cols] = w
    v = v.reshape(E, rows, G, group)
    scales = bf16(np.abs(v).max(-1) * np.float32(1.0 / 6.0))
    s = scales[..., None]
    a = np.divide(np.abs(v), s, out=np.zeros_like(v), where=s > 0)
    code = np.zeros(a.shape, np.uint8)
    for bound, inclusive in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5, 0)):
        code += (a >= bound) if inclusive else (a > bound)
    code += 8 * np.signbit(v).astype(np.uint8)
    return code.reshape(E, rows, -1)[:, :, :cols], scales


def dequantize(codes, scales, group):
    v = MAG[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    at = np.arange(codes.shape[2]) // group
    return v * scales.astype(np.float64)[:, :, at]


def pack(codes):
    """The storage of include/moe.h: byte array of the codes."""
    E, rows, cols = codes.shape
    KC = -(-cols // 128)
    c = np.zeros((E, rows, KC * 128), np.uint32)
    c[:, :, :cols] = codes
    words = np.zeros((E, KC, rows // 8, 128), np.uint32)
    for r in range(8):
        for col in range(128):
            words[:, :, :, (col % 32 // 8 * 8 + r) * 4 + col // 32] |= (
                c[:, r::8, col::128].transpose(0, 2, 1) << np.uint32(4 * (col % 8)))
    return words.reshape(-1).view(np.uint8)


def pack_scales(scales, cols, group):
    """The storage of include/moe.h: [E][KC][rows][128 / group]."""
    E, rows, G = scales.shape
    KC, per = -(-cols // 128), 128 // group
    out = np.zeros((E, rows, KC * per), np.float32)
    out[:, :, :G] = scales
    return out.reshape(E, rows, KC, per).transpose(0, 2, 1, 3)


def silu(v):
    return v / (1.0 + np.exp(-v))


def ffn(x, w1, b1, w2, b2, gated):
    """y of rows x of one expert (64 bits) and a bound on what the kernels' arithmetic adds: fp32
    sums (each addition may truncate: a whole step, 2 U) with one scale product a group, the
    activation's evaluation, bf16 rounding of the activation and of y."""
    f = w2.shape[1]
    pre = x @ w1.T
    dpre = (np.abs(x) @ np.abs(w1).T) * (x.shape[1] + 40) * 2 * U
    if gated:
        g, u = pre[:, :f], pre[:, f:]
        dg, du = dpre[:, :f], dpre[:, f:]
        h = silu(g) * u
        # |silu'| <= 1.1; exp's argument carries |g| U, its value a few U
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + np.abs(h) * (np.abs(g) + 12) * 2 * U
    else:
        pre, dpre = pre + b1, dpre + 2 * U * (np.abs(pre) + np.abs(b1))
        h = silu(pre)
        dh = 1.1 * dpre + np.abs(h) * (np.abs(pre) + 12) * 2 * U
    dh = dh + BF * (np.abs(h) + dh)
    y = h @ w2.T
    aw = np.abs(w2).T
    dy = dh @ aw + ((np.abs(h) + dh) @ aw) * (f + 40) * 2 * U
    if not gated:
        y = y + b2
        dy = dy + 2 * U * (np.abs(y) + np.abs(b2))
    return y, dy + BF * (np.abs(y) + dy) + 1e-38
