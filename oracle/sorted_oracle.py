"""CPU oracle of the calls around rows sorted by expert: the sort itself, the way
there and back, the gradients, and products with 4-bit weights.

TEST INFRASTRUCTURE ONLY, as moe_oracle.py: plain NumPy in float64, no code shared
with the library.  Each function is pinned by a closed form, a brute force or
differences in tests/test_oracle_sorted.py."""
from __future__ import annotations

import numpy as np


def sort_pairs(ids, E):
    """ids [T, k] -> offsets [E + 1], perm [live], rows [T, k] (-1: id outside [0, E))."""
    flat = np.asarray(ids).reshape(-1)
    perm = [p for e in range(E) for p in np.flatnonzero(flat == e)]
    rows = np.full(flat.size, -1, np.int32)
    rows[perm] = np.arange(len(perm))
    offsets = np.concatenate([[0], np.cumsum([np.sum(flat == e) for e in range(E)])])
    return offsets.astype(np.int32), np.array(perm, np.int32), rows.reshape(np.shape(ids))


def unpermute(ys, rows, w=None, base=None):
    """(out, the sum of the terms' magnitudes), both [T, H]."""
    M, H = ys.shape
    T, k = rows.shape
    out = np.zeros((T, H)) if base is None else np.array(base, np.float64)
    mag = np.abs(out)
    for t in range(T):
        for r in range(k):
            if 0 <= rows[t, r] < M:
                term = ys[rows[t, r]] * (1.0 if w is None else w[t, r])
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def unpermute_grad(gout, ys, rows, w, gys):
    """(gys with the pairs' rows replaced, gw, the sum of gw's terms' magnitudes)."""
    gys, gw, mag = np.array(gys, np.float64), np.zeros(rows.shape), np.zeros(rows.shape)
    for t, r in np.ndindex(*rows.shape):
        i = rows[t, r]
        if 0 <= i < len(ys):
            gys[i] = gout[t] * (1.0 if w is None else w[t, r])
            gw[t, r] = np.dot(gout[t], ys[i])
            mag[t, r] = np.dot(np.abs(gout[t]), np.abs(ys[i]))
    return gys, gw, mag


LOWEST = -float.fromhex("0x1.fep127")


def scores(logits, scoring):
    """Scores [T, E] with masked logits (NaN, or down from bf16's lowest value) at 0."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x) | (x <= LOWEST), -np.inf, x)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-x))
    top = x.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(x == top, 1.0, np.exp(x - top))
    e = np.where(x == -np.inf, 0.0, e)
    return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)


def route_grad(logits, ids, w, g, scoring, renorm):
    """(glogits [T, E], the magnitudes of what is added up)."""
    s = scores(logits, scoring)
    away = scores(-np.asarray(logits, np.float64), "sigmoid")  # 1 - s without its cancellation near 1
    out, mag = np.zeros_like(s), np.zeros_like(s)
    for t in range(len(s)):
        live = [i for i in range(ids.shape[1]) if 0 <= ids[t, i] < s.shape[1] and w[t, i] != 0]
        total = sum(w[t, i] for i in live)
        m = sum(g[t, i] * w[t, i] for i in live) / total if renorm and total != 0 else 0.0
        if scoring == "softmax" and not renorm:
            out[t] = -s[t] * sum(g[t, i] * w[t, i] for i in live)
            mag[t] = np.abs(out[t])
        for i in live:
            e = ids[t, i]
            d = w[t, i] * (g[t, i] - m) * (away[t, e] if scoring == "sigmoid" else 1.0)
            out[t, e] += d
            mag[t, e] += abs(d)
    return out, mag


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def q4_matrix(codes, scales, group, code, zeros=None):
    """codes [R, K/2] bytes, scales [R, K/group] (values), zeros [R, K/group] or None -> [R, K]."""
    q = np.stack([codes & 15, codes >> 4], -1).reshape(len(codes), -1).astype(int)
    if code == "fp4":
        v = np.where(q < 8, 1.0, -1.0) * E2M1[q & 7]
    else:
        z = 8 if zeros is None else np.repeat(zeros.astype(int), group, axis=1)
        v = (q - z).astype(np.float64)
    return v * np.repeat(scales, group, axis=1)


def q4_product(x, W, act, roundings):
    """(y, its tolerance before the last rounding): every product's way to its sum passes at
    most `roundings` roundings of 2^-24 of the terms' magnitudes."""
    y, err = x @ W.T, roundings * 2.0 ** -24 * (np.abs(x) @ np.abs(W).T)
    if act == "none":
        return y, err
    N = len(W) // 2
    g, u, dg, du = y[:, :N], y[:, N:], err[:, :N], err[:, N:]
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
    h = g * s * u
    # silu's slope is at most 1.1; sigmoid and the two products in at most 12 roundings
    return h, 1.1 * dg * (np.abs(u) + du) + np.abs(g * s) * du + 12 * 2.0 ** -24 * np.abs(h)
