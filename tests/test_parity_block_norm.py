"""GPU parity of the norms of narrow rows, and of gates far from 0, where a sigmoid's relative error
shows, against float64.

u = 2^-24 is half a step of fp32.  1 / (1 + e^-g): the exponential is within a
step (2 u) of its value and corrected with one rounding, the correction's own parts
less than u together, 1 + e one rounding, the reciprocal within a step (2 u): 7 u, 8
with second-order terms; alpha, the product with y and the sum with a residual of 0
round once each: 11 u.
Below 2^-126 the reciprocal may give 0."""
import numpy as np
import pytest

from oracle import block_oracle as B
from tests.test_parity_block import U, Guarded, _c, _close, _f64, _norm_out_ref, _torch, _up

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


@pytest.mark.parametrize("T,H", [(1, 512), (7000, 200), (5000, 512), (5000, 600), (2100, 520), (22000, 400), (17000, 512),
                                 (30000, 300)])
def test_narrow_rows_many_at_a_time(gpu_lib, T, H):
    """Rows of fewer chunks than a wavefront has lanes and a little more, on both sides of the
    sizes where a thread takes a second chunk and where workgroups go on over the rows."""
    torch = _torch()
    rng = np.random.default_rng(T + H)
    eps = float(np.float32(1e-5))
    y, res = _up(rng.standard_normal((T, H)), "bf16", 1), _up(rng.standard_normal((T, H)) * 2, "bf16")
    gate, w = _up(rng.standard_normal(H), "bf16"), _up(rng.standard_normal(H), "bf16")
    norm = gpu_lib.make_norm(H, 1e-5, pre=w, post=w, gate="channel", alpha=0.5)
    out, nout, n_in = Guarded((T, H), "bf16"), Guarded((T, H), "f32", 1), Guarded((T, H), "f32")
    gpu_lib.moe_norm_out(norm, y, res, gate, out.t, norm, nout.t)
    gpu_lib.moe_norm_in(norm, y, n_in.t)
    torch.cuda.synchronize()
    ref, tol, nref, ntol = _norm_out_ref(_f64(y), _f64(res), _f64(gate), _f64(w), _f64(w), "channel", "none", 0.5, True,
                                         0.0, eps, torch.bfloat16, torch.float32)
    _close(_f64(out.check()), ref, tol, "out")
    _close(_f64(nout.check()), nref, ntol, "next")
    ref = B.rms(_f64(y), _f64(w), eps)
    _close(_f64(n_in.check()), ref, np.abs(ref) * (_c(H) + 1) * U, "norm_in")
