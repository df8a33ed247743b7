"""Pins of the block oracle (no GPU): closed forms, brute force and agreement
with the routing oracle where both define the same thing."""
import itertools
import math

import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O


def test_rms_closed_form():
    z = np.array([[3.0, 4.0, 0.0, 0.0], [1.0, -1.0, 1.0, -1.0]])
    got = B.rms(z, np.array([1.0, 2.0, 3.0, 4.0]), 0.0)
    assert np.allclose(got, [[1.2, 3.2, 0.0, 0.0], [1.0, -2.0, 3.0, -4.0]], rtol=0, atol=1e-15)
    assert np.allclose(B.rms(z, np.zeros(4), 0.0, offset=1.0), B.rms(z, None, 0.0))
    assert np.allclose((B.rms(z, None, 0.0) ** 2).mean(axis=1), 1.0)


def test_norm_out_closed_form():
    y, r = np.array([[2.0, -2.0]]), np.array([[10.0, 20.0]])
    assert np.allclose(B.norm_out(y, r, None, 0.0), [[11.0, 19.0]])
    assert np.allclose(B.norm_out(y, r, None, 0.0, gate=[0.0], kind="token", act="sigmoid", alpha=4.0), [[12.0, 18.0]])
    assert np.allclose(B.norm_out(y, r, None, 0.0, gate=[1.0, 0.5], kind="channel", post=False), [[12.0, 19.0]])
    assert np.allclose(B.norm_out(y, r, None, 0.0, gate=[[0.0, 3.0]], kind="full"), [[10.0, 17.0]])


def test_route_groups_without_groups_is_softmax_topk():
    lg = np.random.default_rng(3).standard_normal((20, 64)).astype(np.float32)
    ids, w = B.route_groups(lg, 6, scoring="softmax")
    oids, ow = O.route(lg, 6)
    assert np.array_equal(ids, oids) and np.allclose(w, ow, rtol=1e-14)


@pytest.mark.parametrize("score", ["max", "top2"])
def test_route_groups_brute_force(score):
    """Every set of groups and every set of experts, compared by value."""
    rng = np.random.default_rng(5)
    E, G, tg, k = 12, 4, 2, 3
    for _ in range(30):
        lg, bias = rng.standard_normal(E), 0.3 * rng.standard_normal(E)
        ids, w = B.route_groups(lg[None], k, bias=bias, groups=G, topk_groups=tg, group_score=score, scale=2.0)
        s = 1 / (1 + np.exp(-lg))
        c = s + bias
        value = [np.sort(c[3 * g:3 * g + 3])[::-1][:1 if score == "max" else 2].sum() for g in range(G)]
        gset = max(itertools.combinations(range(G), tg), key=lambda S: sum(value[g] for g in S))
        pool = [e for e in range(E) if e // 3 in gset]
        best = max(itertools.combinations(pool, k), key=lambda S: sum(c[e] for e in S))
        assert set(ids[0].tolist()) == set(best)
        assert np.allclose(w[0], 2.0 * s[ids[0]] / s[list(best)].sum(), rtol=1e-12)
        assert np.all(np.diff(w[0]) <= 0)


def test_route_groups_masks_and_ties():
    inf = math.inf
    ids, w = B.route_groups(np.full((1, 6), -inf), 2)
    assert ids[0].tolist() == [0, 1] and w[0].tolist() == [0.0, 0.0]
    ids, w = B.route_groups(np.array([[-inf, 1.0, np.nan, -inf]]), 3, scoring="softmax")
    assert ids[0].tolist() == [1, 0, 2] and w[0].tolist() == [1.0, 0.0, 0.0]
    ids, w = B.route_groups(np.zeros((1, 8)), 3, groups=4, topk_groups=2)
    assert ids[0].tolist() == [0, 1, 2] and np.allclose(w[0], 1 / 3)
    ids, w = B.route_groups(np.array([[inf, 0.0, inf, 0.0]]), 3, scoring="softmax", renorm=False)
    assert ids[0].tolist() == [0, 2, 1] and w[0].tolist() == [0.5, 0.5, 0.0]
    # a type's lowest value masks as -inf does, whatever the bias
    low = [float(np.finfo(np.float32).min), -(2.0 - 2.0 ** -7) * 2.0 ** 127, -9.0, -1e38]
    ids, w = B.route_groups(np.array([low]), 4, bias=[9.0, 9.0, 0.0, 0.0], renorm=False)
    assert ids[0].tolist() == [2, 0, 1, 3] and w[0, 0] > 0 and not w[0, 1:].any()
    # a group with one unmasked expert is worth that expert, not -inf
    ids, _ = B.route_groups(np.array([[-inf, 3.0, -inf, -inf, -1.0, -inf]]), 1, groups=3, topk_groups=1)
    assert ids[0].tolist() == [1]
    # the bias steers the choice, the weight stays the score
    ids, w = B.route_groups(np.array([[2.0, 0.0]]), 1, bias=[0.0, 5.0], renorm=False)
    assert ids[0].tolist() == [1] and w[0].tolist() == [0.5]


def test_lora_closed_form():
    x = np.array([[1.0, 2.0], [1.0, 2.0], [1.0, 2.0]])
    a = np.array([[[1.0, 1.0], [0.0, 1.0]], [[2.0, 0.0], [9.0, 9.0]]])
    b = np.array([[[1.0, 0.0], [0.0, 1.0], [1.0, 1.0]], [[1.0, 9.0], [2.0, 9.0], [3.0, 9.0]]])
    out, _, _ = B.lora_add(x, [0, 1, -1], np.ones((3, 3)), a, b, scale=[1.0, 0.5], ranks=[2, 1])
    assert np.allclose(out, [[4.0, 3.0, 6.0], [2.0, 3.0, 4.0], [1.0, 1.0, 1.0]])
