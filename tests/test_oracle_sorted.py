"""The oracle of the sorted-rows calls against closed forms, brute force and differences (CPU)."""
import numpy as np
import pytest

from oracle import block_oracle as BO
from oracle import moe_oracle as O
from oracle import sorted_oracle as S


def test_sort_is_stable_and_drops_ids_outside():
    ids = np.array([[2, 0], [-1, 2], [0, 5], [1, 2]])
    offsets, perm, rows = S.sort_pairs(ids, 4)
    assert offsets.tolist() == [0, 2, 3, 6, 6]
    assert perm.tolist() == [1, 4, 6, 0, 3, 7]
    assert rows.tolist() == [[3, 0], [-1, 4], [1, -1], [2, 5]]


@pytest.mark.parametrize("weights", [True, False])
def test_unpermute_and_its_gradient_by_differences(weights):
    rng = np.random.default_rng(0)
    T, k, H, E = 5, 3, 4, 6
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)])
    ids[1, 2] = -1
    rows = S.sort_pairs(ids, E)[2]
    ys, w, g = rng.standard_normal((T * k, H)), rng.standard_normal((T, k)), rng.standard_normal((T, H))
    w = w if weights else None
    loss = lambda y, v: float((S.unpermute(y, rows, v)[0] * g).sum())  # noqa: E731
    gys, gw, _ = S.unpermute_grad(g, ys, rows, w, np.zeros_like(ys))
    for i in np.ndindex(*ys.shape):
        d = np.zeros_like(ys)
        d[i] = 0.5
        assert abs(loss(ys + d, w) - loss(ys - d, w) - gys[i]) < 1e-12
    if weights:
        for i in np.ndindex(*w.shape):
            d = np.zeros_like(w)
            d[i] = 0.5
            assert abs(loss(ys, w + d) - loss(ys, w - d) - gw[i]) < 1e-12
    # without weights it is the gradient of the copy into the order
    x, gx = rng.standard_normal((T, H)), S.unpermute(ys, rows)[0]
    perm = S.sort_pairs(ids, E)[1]
    assert abs((x[perm // k] * ys[:len(perm)]).sum() - (x * gx).sum()) < 1e-10


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_by_differences(scoring, renorm):
    rng = np.random.default_rng(1)
    T, E, k, scale = 3, 9, 4, 1.7
    x, g = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    ids, w = BO.route_groups(x, k, scoring=scoring, renorm=renorm, scale=scale)

    def weights(y):  # the same picks
        s = np.take_along_axis(S.scores(y, scoring), ids, 1)
        return scale * (s / s.sum(1, keepdims=True) if renorm else s)
    assert np.allclose(weights(x), w, atol=1e-14)
    got = S.route_grad(x, ids, w, g, scoring, renorm)[0]
    h = 1e-5
    for i in np.ndindex(T, E):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((g * (weights(x + d) - weights(x - d))).sum() / (2 * h) - got[i]) < 1e-8


def test_route_grad_masks_weigh_nothing():
    x = np.array([[1.0, -np.inf, np.nan, 0.5]])
    ids, w = np.array([[0, 1, 2, -1]]), np.array([[1.0, 0.0, 0.0, 0.0]])
    g = np.array([[3.0, np.inf, np.nan, np.nan]])
    for scoring in ("sigmoid", "softmax"):
        assert np.isfinite(S.route_grad(x, ids, w, g, scoring, True)[0]).all()
        assert np.isfinite(S.route_grad(x, ids, w, g, scoring, False)[0]).all()


def test_q4_matrix_matches_the_records():
    """A record's w1 and w3 together, and its w2, are 4-bit matrices with E8M0 scales per 32."""
    from mxfp4_routed_expert_renorm_amd import workloads as W
    H, I = 64, 96
    rec = W.fp4_record(3, 0, 0, H, I)
    n = H * I // 2
    sc = 2.0 ** (rec[3 * n:].astype(np.float64) - 127)
    both = S.q4_matrix(rec[:2 * n].reshape(2 * I, H // 2), sc[:2 * H * I // 32].reshape(2 * I, -1), 32, "fp4")
    down = S.q4_matrix(rec[2 * n:3 * n].reshape(H, I // 2), sc[2 * H * I // 32:].reshape(H, -1), 32, "fp4")
    x = np.random.default_rng(2).standard_normal((3, H))
    h, _ = S.q4_product(x, both, "swiglu", 0)
    y, _ = S.q4_product(h, down, "none", 0)
    ref = O.layer_forward(x, np.zeros((3, 1), np.int32), np.ones((3, 1)), lambda e: rec, H, I)
    assert np.allclose(y, ref, rtol=1e-12, atol=1e-12)


def test_q4_integers():
    codes = np.array([[0x10, 0xf8] * 8], np.uint8)  # 0, 1, 8, 15
    W = S.q4_matrix(codes, np.array([[2.0]]), 32, "int4")
    assert W[0, :4].tolist() == [-16.0, -14.0, 0.0, 14.0]
    W = S.q4_matrix(codes, np.array([[2.0]]), 32, "int4", np.array([[1]], np.uint8))
    assert W[0, :4].tolist() == [-2.0, 0.0, 14.0, 28.0]
