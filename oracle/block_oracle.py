"""CPU oracle of the operators around the experts: norms before and after a
block, expert choice by scores, bias and groups, and many requests' low-rank
adapters.

TEST INFRASTRUCTURE ONLY, as moe_oracle.py: plain NumPy in float64, no code
shared with the library.  Each function is pinned by a closed form or a brute
force in tests/test_oracle_block.py."""
from __future__ import annotations

import numpy as np


def rms(z, w, eps, offset=0.0):
    """z [T, H] over the root of its rows' mean square, times (offset + w); w None: times 1."""
    z = np.asarray(z, np.float64)
    n = z / np.sqrt((z * z).mean(axis=1, keepdims=True) + eps)
    return n if w is None else n * (offset + np.asarray(w, np.float64))


def gate_factor(gate, kind, act, T, H):
    """The gate's factor [T, H]: kind none, channel [H], token [T] or full [T, H]."""
    if kind == "none":
        return np.ones((T, H))
    g = np.asarray(gate, np.float64)
    if act == "sigmoid":
        with np.errstate(over="ignore"):
            g = 1.0 / (1.0 + np.exp(-g))
    g = g[:, None] if kind == "token" else g
    return np.broadcast_to(g, (T, H)).copy()


def norm_out(y, residual, post_w, eps, gate=None, kind="none", act="none", alpha=1.0, post=True, offset=0.0):
    """residual + alpha * gate * RMS(y; post_w), unrounded."""
    y = np.asarray(y, np.float64)
    z = rms(y, post_w, eps, offset) if post else y
    return np.asarray(residual, np.float64) + alpha * gate_factor(gate, kind, act, *y.shape) * z


def route_groups(logits, k, scoring="sigmoid", bias=None, groups=1, topk_groups=None, group_score="top2",
                 renorm=True, scale=1.0):
    """One token at a time: scores, choices, the groups that stay, the picks, their weights.

    A logit of NaN, or down from bf16's lowest value, and a choice of -inf or NaN
    mask their expert: in no group's value, picked last (lower ids first), weight 0."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    topk_groups = groups if topk_groups is None else topk_groups
    size = E // groups
    ids, w = np.empty((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        l = [float(v) if v > -(2.0 - 2.0 ** -7) * 2.0 ** 127 else -np.inf for v in logits[t]]
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):  # an exponential past the range: a score of 0
                s = [0.0 if v == -np.inf else float(1.0 / (1.0 + np.exp(-v))) for v in l]
        else:
            top = max(l)
            e = [0.0 if v == -np.inf else 1.0 if v == top else np.exp(v - top) for v in l]
            total = sum(e)
            s = [v / total if total > 0 else 0.0 for v in e]
        c = []
        for e in range(E):
            v = s[e] if bias is None else s[e] + float(bias[e])
            c.append(-np.inf if l[e] == -np.inf or np.isnan(v) else v)
        value = []
        for g in range(groups):
            live = sorted((v for v in c[g * size:(g + 1) * size] if v != -np.inf), reverse=True)
            value.append(-np.inf if not live else live[0] if group_score == "max" else sum(live[:2]))
        stay = sorted(range(groups), key=lambda g: (-value[g], g))[:topk_groups]
        cand = [e for e in range(E) if e // size in stay]
        picks = sorted(cand, key=lambda e: (-c[e], e))[:k]
        weight = {e: (0.0 if c[e] == -np.inf else s[e]) for e in picks}
        picks.sort(key=lambda e: (-weight[e], e))
        total = sum(weight.values())
        for r, e in enumerate(picks):
            v = weight[e]
            if renorm:
                v = v / total if total > 0 else 0.0
            ids[t, r], w[t, r] = e, v * scale
    return ids, w


def lora_add(x, ids, base, a, b, scale=None, ranks=None):
    """base + scale * B (A x) per token with its adapter; (out, magnitudes).

    The magnitudes bound rounding errors: |v| and sum |A||x| folded through |B|."""
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    T, (num, r, _), N = x.shape[0], a.shape, b.shape[1]
    out = np.zeros((T, N)) if base is None else np.array(base, np.float64)
    through_x, through_v = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        i = int(ids[t])
        if not 0 <= i < num:
            continue
        n = r if ranks is None else max(0, min(int(ranks[i]), r))
        s = 1.0 if scale is None else float(scale[i])
        A, B = a[i, :n], b[i, :, :n]
        v = s * (A @ x[t])
        out[t] += B @ v
        through_x[t] = np.abs(B) @ (abs(s) * (np.abs(A) @ np.abs(x[t])))
        through_v[t] = np.abs(B) @ np.abs(v)
    return out, through_x, through_v
