"""GPU parity of moe_route_groups where double precision decides: weights to one
rounding, and groups whose best scores are equal in double but not as logits."""
import numpy as np
import pytest

from oracle import block_oracle as B
from tests.test_parity_block import U, Guarded, _close, _f64, _torch, _up

pytestmark = pytest.mark.gpu


def _route(gpu_lib, logits, k, lt="f32", bias=None, **kw):
    torch = _torch()
    lg = _up(logits, lt)
    b = None if bias is None else _up(bias, "f32")
    ids, w = Guarded((lg.shape[0], k), "i32"), Guarded((lg.shape[0], k), "f32")
    gpu_lib.moe_route_groups(gpu_lib.make_router(lg.shape[1], k, **kw), lg, b, ids.t, w.t)
    torch.cuda.synchronize()
    want_ids, want_w = B.route_groups(_f64(lg), k, bias=None if b is None else _f64(b), **kw)
    return ids.check().cpu().numpy(), _f64(w.check()), want_ids, want_w


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (300, 6), (512, 8), (1024, 32)])
def test_route_weights_to_one_rounding(gpu_lib, E, k, scoring):
    """Scores, their sums and the scale in double precision: an exponential, a sum of
    E positive terms and a division, off by less than (E + 8) 2^-53 together, then
    one rounding to fp32, 2^-24 of the value (half of 2^-149 below 2^-126)."""
    rng = np.random.default_rng(E)
    for renorm in (False, True):
        for std in (0.3, 1.5, 6.0):
            for kw in (dict(), dict(groups=4, topk_groups=2, group_score="max"), dict(groups=4, topk_groups=3)):
                if kw and kw["topk_groups"] * E // 4 < k:
                    continue
                lg = std * rng.standard_normal((33, E))
                lg[5, ::3] = -np.inf
                got, w, want, ww = _route(gpu_lib, lg, k, scoring=scoring, renorm=renorm, scale=2.5, **kw)
                assert np.array_equal(got, want), kw
                _close(w, ww, np.abs(ww) * (U + (E + 8) * 2.0 ** -53) + 2.0 ** -150, f"weights {renorm} {std} {kw}")


@pytest.mark.parametrize("renorm", [True, False])
def test_route_groups_tied_in_double_but_not_as_logits(gpu_lib, renorm):
    """Softmax, groups by their best score: best logits within the rounding of a
    double exponential are equal scores, and the lower group stays."""
    tiny = 1e-20
    best = [  # per row, the best logit of each of four groups
        (-tiny, 0.0, 0.0, -3.0), (0.0, 0.0, tiny, -3.0), (-2.0, -tiny, 0.0, 0.0), (-tiny, 0.0, -tiny, 0.0),
        (0.0, tiny, 0.0, tiny), (-3.0, -2 * tiny, -tiny, 0.0), (0.0, 0.0, 0.0, 0.0), (-1e-6, 0.0, 0.0, 0.0),
        (0.0, 0.0, 1e-6, -1e-6), (1.0, 1.0, 1.0, 1.0 + 2.0 ** -23), (1e-30, -1e-30, 0.0, 0.0)]
    lg = np.full((len(best), 32), -5.0, np.float32)
    for t, row in enumerate(best):
        lg[t, 3::8] = row
    for kept in (1, 2, 3):
        for k in (1, 4):
            got, _, want, _ = _route(gpu_lib, lg, k, scoring="softmax", groups=4, topk_groups=kept, group_score="max",
                                     renorm=renorm)
            assert np.array_equal(got, want), (kept, k, np.argwhere((got != want).any(1)).ravel())
