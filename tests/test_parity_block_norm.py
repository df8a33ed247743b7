"""GPU parity of the norms' gates far from 0, where a sigmoid's relative error
shows, against float64.

u = 2^-24 is half a step of fp32.  1 / (1 + e^-g): the exponential is within a
step (2 u) of its value and corrected with one rounding, the correction's own parts
less than u together, 1 + e one rounding, the reciprocal within a step (2 u): 7 u, 8
with second-order terms; alpha, the product with y and the sum with a residual of 0
round once each: 11 u.
Below 2^-126 the reciprocal may give 0."""
import numpy as np
import pytest

from tests.test_parity_block import U, Guarded, _close, _f64, _torch, _up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(3, 4096), (700, 2047), (1200, 4096)])
@pytest.mark.parametrize("kind", ["channel", "token", "full"])
def test_sigmoid_gates_far_from_zero(gpu_lib, T, H, kind, gt):
    torch = _torch()
    rng = np.random.default_rng(T)
    gate = _up(rng.uniform(-86.0, 30.0, {"channel": (H,), "token": (T,), "full": (T, H)}[kind]), gt)
    y, res = _up(rng.uniform(0.5, 2.0, (T, H)), "f32"), torch.zeros(T, H, device="cuda")
    out = Guarded((T, H), "f32")
    gpu_lib.moe_norm_out(gpu_lib.make_norm(H, gate=kind, gate_act="sigmoid", alpha=0.75), y, res, gate, out.t)
    torch.cuda.synchronize()
    g = _f64(gate)
    ref = 0.75 * _f64(y) / (1.0 + np.exp(-(g[:, None] if kind == "token" else g)))
    _close(_f64(out.check()), ref, 11 * U * ref + 2.0 ** -125, f"gate {kind}")


def test_sigmoid_gates_at_the_ends(gpu_lib):
    """Infinite, NaN and very large gates."""
    torch = _torch()
    gate = torch.tensor([float("inf"), -float("inf"), float("nan"), 200.0, -200.0, 3e38, -3e38, 0.0], device="cuda")
    y, res, out = torch.ones(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda"), Guarded((4, 8), "f32")
    gpu_lib.moe_norm_out(gpu_lib.make_norm(8, gate="channel", gate_act="sigmoid"), y, res, gate, out.t)
    torch.cuda.synchronize()
    got = out.check().cpu()
    assert bool(got[:, 2].isnan().all())
    want = torch.tensor([1.0, 0.0, 1.0, 0.0, 1.0, 0.0, 0.5])
    assert torch.equal(got[:, [0, 1, 3, 4, 5, 6, 7]], want.expand(4, 7))
