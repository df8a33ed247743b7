"""GPU parity of the products with 4-bit weights where there are many rows, of every scale
byte, and of the few-row form's larger grids, against the float64 oracle.

The tolerances are those of test_parity_q4.py."""
import numpy as np
import pytest

from tests.test_parity_block import Guarded, _close, _f64, _torch, _up
from tests.test_parity_q4 import FORMS, Weights, _grouped
from tests.test_parity_sorted import _i32

pytestmark = pytest.mark.gpu


# inputs in 5 and 13 blocks of 32 (scales that start anywhere), 6 (at even places), 8 and 24
@pytest.mark.parametrize("K,group", [(160, 32), (192, 32), (192, 64), (256, 128), (416, 32), (768, 32), (768, 256)])
@pytest.mark.parametrize("code,scale,zeros", FORMS)
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f32")])
def test_q4_linear_tiles(gpu_lib, K, group, code, scale, zeros, xt, yt):
    torch = _torch()
    rng = np.random.default_rng(K + group)
    for T, N, act in ((1300, 1301, "none"), (3200, 1400, "none"), (1100, 750, "swiglu")):
        w = Weights(gpu_lib, rng, 1, N, K, group, code, scale, zeros, act)
        x = _up(rng.standard_normal((T, K)) / K ** 0.5, xt)
        y = Guarded((T, N), yt, N % 2)
        gpu_lib.moe_q4_linear(w.q4, x, y.t)
        torch.cuda.synchronize()
        _close(_f64(y.check()), *w.product(_f64(x), 0, yt), f"q4 {T} x {N} x {K}")


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("code,scale,zeros", FORMS[:3])
def test_q4_linear_rows_of_x_anywhere(gpu_lib, shift, xt, code, scale, zeros):
    """x and y off the 16 bytes, with as many rows."""
    torch = _torch()
    rng = np.random.default_rng(shift)
    T, N, K = 1300, 1301, 256
    w = Weights(gpu_lib, rng, 1, N, K, 32, code, scale, zeros, "none")
    x = _up(rng.standard_normal((T, K)) / K ** 0.5, xt, shift)
    y = Guarded((T, N), "bf16", 1)
    gpu_lib.moe_q4_linear(w.q4, x, y.t)
    torch.cuda.synchronize()
    _close(_f64(y.check()), *w.product(_f64(x), 0, "bf16"), f"x off by {shift}")


@pytest.mark.parametrize("counts", [[700, 0, 1, 129, 500, 3], [64, 65] * 12, [0, 1400, 0],
                                    [0] * 66 + [1300, 1, 127, 128]], ids=lambda c: f"{len(c)}m{sum(c)}r")
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("code,scale", [("int4", "bf16"), ("fp4", "e8m0"), ("fp4", "f32")])
def test_q4_grouped_tiles(gpu_lib, counts, xt, yt, code, scale):
    rng = np.random.default_rng(len(counts))
    for K, N, group, act, first, behind in ((160, 750, 32, "swiglu", 2, 130), (256, 1301, 128, "none", 0, 0),
                                            (256, 1301, 32, "none", 3, 1)):
        w = Weights(gpu_lib, rng, len(counts), N, K, group, code, scale, code == "int4", act, apart=len(counts) % 3)
        _grouped_aligned(gpu_lib, rng, w, counts, xt, yt, behind, first)


def _grouped_aligned(lib, rng, w, counts, xt, yt, behind, first):
    torch = _torch()
    offsets = first + np.concatenate([[0], np.cumsum(counts)])
    P = int(offsets[-1]) + behind
    x = rng.standard_normal((P, w.K)) / w.K ** 0.5
    x[:first], x[P - behind:] = np.nan, np.nan
    x, y = _up(x, xt), Guarded((P, w.N), yt, 1)
    lib.moe_q4_grouped(w.q4, x, _i32(offsets), y.t)
    torch.cuda.synchronize()
    got, x64 = _f64(y.check()), _f64(x)
    assert (got[:first] == 77).all() and (got[P - behind:] == 77).all(), "rows outside the matrices'"
    for e in range(w.num):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            ref, tol = w.product(x64[lo:hi], e, yt)
            _close(got[lo:hi], ref, tol, f"matrix {e} rows {lo}..{hi}")


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("code,scale,zeros", FORMS)
def test_q4_few_rows_of_a_long_matrix(gpu_lib, xt, code, scale, zeros):
    """One workgroup a compute unit, and more."""
    torch = _torch()
    rng = np.random.default_rng(11)
    for T, N, K, group in ((3, 4200, 4128, 32), (20, 2100, 2048, 128), (2, 4097, 1056, 1056)):
        w = Weights(gpu_lib, rng, 1, N, K, group, code, scale, zeros, "none")
        x = _up(rng.standard_normal((T, K)) / K ** 0.5, xt)
        y = Guarded((T, N), "f32")
        gpu_lib.moe_q4_linear(w.q4, x, y.t)
        torch.cuda.synchronize()
        _close(_f64(y.check()), *w.product(_f64(x), 0, "f32"), f"{T} x {N} x {K}")
    w = Weights(gpu_lib, rng, 30, 160, 1024, 256, code, scale, zeros, "swiglu")
    _grouped(gpu_lib, rng, w, [1, 0, 20] * 10, xt, "f32")


@pytest.mark.parametrize("T", [128, 3328])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("code,group", [("fp4", 32), ("fp4", 64), ("fp4", 128), ("int4", 32), ("int4", 128)])
def test_q4_every_scale_byte(gpu_lib, T, xt, code, group):
    """Unit rows of x read each code under each of the 256 scale bytes, exactly: the smallest
    powers are subnormal, the largest codes of the largest ones pass fp32's range, 255 is NaN."""
    torch = _torch()
    K, N = 128, 512
    codes = np.random.default_rng(0).integers(0, 256, (N, K // 2), dtype=np.uint8)
    raw = (np.arange(N)[:, None] + 64 * np.arange(K // group)[None]).astype(np.uint8)
    q4 = gpu_lib.make_q4(torch.from_numpy(codes).cuda(), torch.from_numpy(raw).cuda(), code=code)
    pair = np.stack([codes & 15, codes >> 4], -1).reshape(N, K).astype(int)
    if code == "fp4":
        value = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])[pair & 7] * np.where(pair & 8, -1.0, 1.0)
    else:
        value = pair - 8.0
    s = np.where(raw == 255, np.nan, 2.0 ** (raw.astype(np.float64) - 127)).repeat(group, 1)
    with np.errstate(over="ignore"):
        want = (value * s).astype(np.float32).T
    x = torch.eye(K, device="cuda").repeat(T // K, 1).to(torch.bfloat16 if xt == "bf16" else torch.float32)
    y = torch.empty(T, N, device="cuda")
    gpu_lib.moe_q4_linear(q4, x.contiguous(), y)
    got = y.cpu().numpy()[:K]
    # a row of x has zeros for the other inputs: where their weights are not finite, no value is right
    big = ~np.isfinite(value * s).T | (np.abs(value * s).T > float(np.finfo(np.float32).max))
    clean = ~big.any(0)
    assert clean.sum() > N // 3
    assert np.array_equal(got[:, clean], want[:, clean])
    for r in range(1, T // K):
        assert torch.equal(y[:K, torch.from_numpy(clean).cuda()], y[r * K:(r + 1) * K, torch.from_numpy(clean).cuda()])
    assert not np.isfinite(got[:, (raw == 255).all(1)]).any()
