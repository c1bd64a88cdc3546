"""Plain 64-bit forms of the MX4 format, its product and the expert layer
(numpy and torch doubles; no code of the library)."""
from __future__ import annotations

import numpy as np
import torch

from _helpers import bits_to_f64

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(bits):
    """BF16 bits [rows, cols] -> (codes uint8 [rows, cols], scale bytes [rows, cols/32])."""
    v = bits_to_f64(bits).reshape(bits.shape[0], -1, 32)
    codes = np.zeros(v.shape, np.uint8)
    scales = np.zeros(v.shape[:2], np.uint8)
    for r in range(v.shape[0]):
        for g in range(v.shape[1]):
            b = v[r, g]
            if not np.all(np.isfinite(b)):
                scales[r, g] = 255
                continue
            m = np.abs(b).max()
            e = -127
            if m > 0:
                e = min(max(int(np.frexp(m)[1]) - 1 - 2, -127), 127)
            scales[r, g] = e + 127
            a = np.minimum(np.abs(b) * 2.0 ** -e, 6.0)
            d = np.abs(a[:, None] - GRID[None, :])
            near = d.min(axis=1)
            # the nearest value; of two equally near ones the even code
            pick = np.array([min((c for c in range(8) if d[i, c] == near[i]), key=lambda c: c & 1) for i in range(32)])
            codes[r, g] = pick + 8 * np.signbit(b)
    return codes.reshape(bits.shape), scales


def pack(codes):
    c = codes.reshape(codes.shape[0], -1, 8).astype(np.uint32)
    return (c << (4 * np.arange(8, dtype=np.uint32))).sum(axis=-1, dtype=np.uint32)


def values(codes, scales):
    """fp64 values of codes [rows, cols] and scale bytes."""
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
        v = np.where(codes >= 8, -1.0, 1.0) * GRID[codes & 7]
        return v * np.repeat(s, 32, axis=1)


def random_weight(g, rows, cols, low=117, high=123):
    """Random codes and scale bytes in [low, high)."""
    return g.integers(0, 16, (rows, cols), dtype=np.uint8), g.integers(low, high, (rows, cols // 32)).astype(np.uint8)


def moe(x, router, gate, up, down, top_k, renorm):
    """The layer in doubles (torch tensors, any device): x [m, H], router [E, H], gate and
    up [E, I, H], down [E, H, I].  Returns (y, ids, err): err bounds |y' - y| of a
    y' whose g and u are fp32 sums, whose h is rounded to BF16 and which is an
    fp32 sum rounded to BF16 (see the derivation below)."""
    m, H = x.shape
    E, I = gate.shape[:2]
    logits = x @ router.t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)[1]
    ids = order[:, :top_k]
    y = torch.zeros_like(x)
    err = torch.zeros_like(x)
    # fp32 sum of n products on the tensor pipe: each of the n / 16 MMAs loses
    # at most 2^-22 of the sum of magnitudes
    gh, gi = (H / 16 + 32) * 2.0 ** -22, (top_k * I / 16 + 32) * 2.0 ** -22
    for t in range(m):
        w = torch.exp(logits[t] - logits[t].max())
        total = w[ids[t]].sum() if renorm else w.sum()
        for e in ids[t].tolist():
            p = w[e] / total
            g, u = gate[e] @ x[t], up[e] @ x[t]
            sg, su = gate[e].abs() @ x[t].abs(), up[e].abs() @ x[t].abs()
            s = g / (1 + torch.exp(-g))
            h = p * s * u
            # |silu'| <= 1.1; 2^-8 |h| is the rounding of h; 2^-18 covers expf,
            # the division, p and the products
            dh = p * (1.1 * gh * sg * u.abs() + (s.abs() + 1.1 * gh * sg) * gh * su) + (2.0 ** -8 + 2.0 ** -18) * h.abs()
            y[t] += down[e] @ h
            err[t] += down[e].abs() @ (dh + gi * h.abs())
    return y, ids, err + 2.0 ** -8 * (y.abs() + err)
