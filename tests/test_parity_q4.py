"""GPU parity of the products with 4-bit weights against the float64 oracle.

Products are exact, so an output's error is the roundings of its sums: a product passes
through at most 32 additions of its matrix instruction, one a later instruction of its
group (three parts of fp32 x: three a 32 inputs), one a later group, and 16 where the
wavefronts' sums meet.  The matrix units may truncate, so each counts double."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import sorted_oracle as S
from mxfp4_routed_expert_renorm_amd import workloads as W
from tests.test_parity_block import U, Guarded, _close, _dt, _f64, _half, _torch, _up
from tests.test_parity_sorted import _i32, _permute

pytestmark = pytest.mark.gpu


def _roundings(K, group):
    return 2 * (32 + 3 * (group // 32) + K // group + 16)


class Weights:
    """num matrices of random codes, with their float64 values."""

    def __init__(self, lib, rng, num, N, K, group, code, scale, zeros, act, apart=0):
        torch = _torch()
        R, G = N * (2 if act == "swiglu" else 1), K // group
        self.codes = rng.integers(0, 256, (num, R, K // 2), dtype=np.uint8)
        self.zeros = rng.integers(0, 16, (num, R, G), dtype=np.uint8) if zeros else None
        if scale == "e8m0":
            raw = rng.integers(117, 126, (num, R, G), dtype=np.uint8)
            self.scales, s = 2.0 ** (raw.astype(np.float64) - 127), torch.from_numpy(raw).cuda()
        else:
            s = _up(0.05 * np.exp(0.5 * rng.standard_normal((num, R, G))), scale)
            self.scales = _f64(s)
        self.group, self.code, self.act, self.num, self.N, self.K = group, code, act, num, N, K
        c = torch.from_numpy(self.codes).cuda()
        if apart:  # matrices that stand apart, as in a bank of records
            far = torch.full((num, R * K // 2 + 16 * apart), 0xEE, dtype=torch.uint8, device="cuda")
            far[:, :R * K // 2] = c.view(num, -1)
            c = far[:, :R * K // 2].unflatten(1, (R, K // 2))
        z = None if self.zeros is None else torch.from_numpy(self.zeros).cuda()
        self.q4 = lib.make_q4(c, s, z, code=code, act=act)

    def matrix(self, e):
        return S.q4_matrix(self.codes[e], self.scales[e], self.group, self.code,
                           None if self.zeros is None else self.zeros[e])

    def product(self, x, e, yt):
        y, err = S.q4_product(x, self.matrix(e), self.act, _roundings(self.K, self.group))
        return y, err + _half(_dt(yt)) * (np.abs(y) + err) + 1e-37


FORMS = [("int4", "bf16", True), ("int4", "f32", False), ("fp4", "e8m0", False), ("fp4", "bf16", False),
         ("int4", "e8m0", True), ("fp4", "f32", False)]


@pytest.mark.parametrize("K,N,group", [(32, 1, 32), (64, 16, 64), (96, 17, 96), (128, 33, 32), (160, 5, 160), (256, 64, 128),
                                       (320, 40, 64), (384, 100, 192), (1024, 130, 1024), (2016, 30, 2016),
                                       (4096, 48, 128), (4128, 20, 32), (8192, 16, 256)])
@pytest.mark.parametrize("code,scale,zeros", FORMS)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_q4_linear(gpu_lib, K, N, group, code, scale, zeros, act):
    torch = _torch()
    rng = np.random.default_rng(K + N)
    w = Weights(gpu_lib, rng, 1, N, K, group, code, scale, zeros, act)
    for n, (T, xt, yt) in enumerate([(1, "bf16", "bf16"), (1, "f32", "f32"), (2, "f32", "bf16"), (17, "bf16", "f32"),
                                     (5, "bf16", "bf16"), (33, "f32", "f32"), (70, "bf16", "bf16")]):
        x = _up(rng.standard_normal((T, K)) / K ** 0.5, xt, n % 3)
        y = Guarded((T, N), yt, n % 3)
        gpu_lib.moe_q4_linear(w.q4, x, y.t)
        torch.cuda.synchronize()
        _close(_f64(y.check()), *w.product(_f64(x), 0, yt), f"q4 T={T} {xt} {yt}")


@pytest.mark.parametrize("T", [15, 16, 31, 64, 65, 127, 128, 129, 200, 257, 513])
@pytest.mark.parametrize("xt,code,act", [("bf16", "int4", "none"), ("f32", "int4", "swiglu"), ("bf16", "fp4", "swiglu"),
                                         ("f32", "fp4", "none")])
def test_q4_linear_many_rows(gpu_lib, T, xt, code, act):
    torch = _torch()
    rng = np.random.default_rng(T)
    for K, N, group in ((416, 70, 32), (512, 300, 128), (320, 129, 64)):
        w = Weights(gpu_lib, rng, 1, N, K, group, code, "bf16", code == "int4", act)
        x = _up(rng.standard_normal((T, K)) / K ** 0.5, xt, 1)
        for yt in ("f32", "bf16"):
            y = Guarded((T, N), yt, 1)
            gpu_lib.moe_q4_linear(w.q4, x, y.t)
            torch.cuda.synchronize()
            _close(_f64(y.check()), *w.product(_f64(x), 0, yt), f"q4 T={T} K={K}")


def _grouped(lib, rng, w, counts, xt, yt, behind=0, first=0):
    """The rows of each matrix against the oracle; the rows before and behind them untouched."""
    torch = _torch()
    offsets = first + np.concatenate([[0], np.cumsum(counts)])
    P = int(offsets[-1]) + behind
    x = rng.standard_normal((P, w.K)) / w.K ** 0.5
    x[:first], x[P - behind:] = np.nan, np.nan
    x, y = _up(x, xt, 1), Guarded((P, w.N), yt, 1)
    lib.moe_q4_grouped(w.q4, x, _i32(offsets), y.t)
    torch.cuda.synchronize()
    got, x64 = _f64(y.check()), _f64(x)
    assert (got[:first] == 77).all() and (got[P - behind:] == 77).all(), "rows outside the matrices'"
    for e in range(w.num):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            ref, tol = w.product(x64[lo:hi], e, yt)
            _close(got[lo:hi], ref, tol, f"matrix {e} rows {lo}..{hi}")


COUNTS = [[1], [0, 3, 0], [16, 1, 15, 0, 17], [0, 0, 0, 64], [5] * 9, [130, 0, 1, 33, 7, 200], [300, 2], [1] * 70,
          [0] * 64 + [3] + [0] * 63 + [2]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}m{sum(c)}r")
@pytest.mark.parametrize("xt,yt,code,scale,act", [("bf16", "bf16", "int4", "bf16", "swiglu"),
                                                  ("f32", "f32", "fp4", "e8m0", "none"),
                                                  ("bf16", "f32", "fp4", "e8m0", "swiglu"),
                                                  ("f32", "bf16", "int4", "f32", "none")])
def test_q4_grouped(gpu_lib, counts, xt, yt, code, scale, act):
    rng = np.random.default_rng(len(counts) + sum(counts))
    for K, N, group in ((160, 50, 32), (512, 24, 128)):
        w = Weights(gpu_lib, rng, len(counts), N, K, group, code, scale, code == "int4", act, apart=len(counts) % 3)
        _grouped(gpu_lib, rng, w, counts, xt, yt, behind=len(counts) % 4, first=0)
    _grouped(gpu_lib, rng, w, counts, xt, yt, behind=3, first=2)


def test_q4_grouped_no_rows_at_all(gpu_lib):
    torch = _torch()
    rng = np.random.default_rng(0)
    w = Weights(gpu_lib, rng, 4, 16, 64, 32, "fp4", "e8m0", False, "none")
    y = Guarded((7, 16), "f32")
    gpu_lib.moe_q4_grouped(w.q4, torch.randn(7, 64, device="cuda"), _i32([0] * 5), y.t)
    assert bool((y.check() == 77).all())
    gpu_lib.moe_q4_grouped(w.q4, torch.empty(0, 64, device="cuda"), _i32([0] * 5), torch.empty(0, 16, device="cuda"))
    gpu_lib.moe_q4_linear(w.q4, torch.empty(0, 64, device="cuda"), torch.empty(0, 16, device="cuda"))


@pytest.mark.parametrize("T", [3, 40, 150])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("code", ["int4", "fp4"])
def test_q4_nonfinite_rows_stay_alone(gpu_lib, T, xt, code):
    torch = _torch()
    rng = np.random.default_rng(7)
    K, N = 256, 40
    w = Weights(gpu_lib, rng, 1, N, K, 64, code, "bf16", False, "none")
    x = _up(rng.standard_normal((T, K)), xt)
    a, b = (torch.empty(T, N, device="cuda") for _ in range(2))
    gpu_lib.moe_q4_linear(w.q4, x, a)
    x[1, 5], x[2, 255] = float("nan"), float("inf")
    if xt == "f32":  # a NaN whose upper half is an infinity's
        x.view(torch.int32)[1, 5] = 0x7F800001
    gpu_lib.moe_q4_linear(w.q4, x, b)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(a[keep], b[keep]) and bool(a.isfinite().all())
    assert bool(b[1].isnan().all()) and not bool(b[2].isfinite().any())


def test_q4_one_weight_at_a_time(gpu_lib):
    """Unit rows of x read single weights back, exactly, at every place of a matrix."""
    torch = _torch()
    rng = np.random.default_rng(8)
    for K, N, group in ((160, 20, 32), (256, 35, 128)):
        for code, scale, zeros in FORMS:
            w = Weights(gpu_lib, rng, 1, N, K, group, code, scale, zeros, "none")
            want = w.matrix(0).T.astype(np.float32)
            for xt in ("bf16", "f32"):
                for T in (K, 7):
                    x = torch.eye(K, device="cuda")[:T].to(_dt(xt)).contiguous()
                    y = torch.empty(T, N, device="cuda")
                    gpu_lib.moe_q4_linear(w.q4, x, y)
                    assert np.array_equal(y.cpu().numpy(), want[:T]), (K, code, scale, xt, T)


def test_q4_fp32_inputs_keep_all_bits(gpu_lib):
    """A single fp32 input of 24 significant bits through a weight of 1."""
    torch = _torch()
    K, N, T = 64, 16, 40
    codes = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device="cuda")  # E2M1 1.0
    q4 = gpu_lib.make_q4(codes, torch.full((N, 2), 127, dtype=torch.uint8, device="cuda"), code="fp4")
    x = torch.zeros(T, K, device="cuda")
    x[torch.arange(T), torch.arange(T)] = torch.randn(T, device="cuda") * torch.logspace(-25, 25, T, device="cuda")
    y = torch.empty(T, N, device="cuda")
    gpu_lib.moe_q4_linear(q4, x, y)
    assert torch.equal(y, x.sum(1, keepdim=True).expand(T, N))


def test_q4_on_expert_records(gpu_lib):
    """The library's own MXFP4 records as matrices that stand apart: routed, sorted,
    multiplied and brought back, against moe_expert_forward's oracle."""
    torch = _torch()
    rng = np.random.default_rng(9)
    T, E, H, I, k = 21, 12, 256, 96, 3
    bank = W.fp4_bank(5, W.S_BANK, E, H, I)
    d, n, m = torch.from_numpy(bank).cuda(), H * I // 2, H * I // 32
    up = gpu_lib.make_q4(d[:, :2 * n].unflatten(1, (2 * I, H // 2)), d[:, 3 * n:3 * n + 2 * m].unflatten(1, (2 * I, -1)),
                         code="fp4", act="swiglu")
    down = gpu_lib.make_q4(d[:, 2 * n:3 * n].unflatten(1, (H, I // 2)), d[:, 3 * n + 2 * m:].unflatten(1, (H, -1)),
                           code="fp4")
    x = _up(rng.standard_normal((T, H)), "f32")
    lg = _up(rng.standard_normal((T, E)), "f32")
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    gpu_lib.moe_route(lg, k, ids, w)
    xs, offsets, perm, rows = _permute(gpu_lib, x, ids, E)
    h, ys, out = (torch.empty(s, device="cuda") for s in ((T * k, I), (T * k, H), (T, H)))
    gpu_lib.moe_q4_grouped(up, xs.t, offsets.t, h)
    gpu_lib.moe_q4_grouped(down, h, offsets.t, ys)
    gpu_lib.moe_unpermute(ys, rows.t, w, None, out)
    torch.cuda.synchronize()
    ref = O.layer_forward(_f64(x), ids.cpu().numpy(), _f64(w), lambda e: bank[e], H, I)
    assert np.linalg.norm(_f64(out) - ref) <= 1e-5 * np.linalg.norm(ref)
    del perm


def test_q4_far_matrices_and_rows(gpu_lib):
    """Codes past 2^32 bytes of a bank, y past 2^31 elements."""
    torch = _torch()
    K, N, num = 8192, 65536, 17
    codes = torch.randint(0, 256, (num, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((num, N, K // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    q4 = gpu_lib.make_q4(codes, scales)
    last = gpu_lib.make_q4(codes[num - 1], scales[num - 1])
    x = torch.randn(2, K, device="cuda").bfloat16()
    y, want = (torch.empty(2, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gpu_lib.moe_q4_grouped(q4, x, _i32([0] * num + [2]), y)
    gpu_lib.moe_q4_linear(last, x, want)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    del codes, scales, q4
    T, K = 33000, 32
    small = gpu_lib.make_q4(torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda"),
                            torch.ones(N, 1, device="cuda"))
    x = torch.randn(T, K, device="cuda").bfloat16()
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    gpu_lib.moe_q4_linear(small, x, y)
    few = torch.empty(40, N, dtype=torch.bfloat16, device="cuda")
    gpu_lib.moe_q4_linear(small, x[-40:].contiguous(), few)
    torch.cuda.synchronize()
    ref = few.float()
    # the two forms group their sums otherwise: a rounding to bf16 may fall to the other side
    assert float(((y[-40:].float() - ref).abs() / ref.abs().clamp_min(0.5)).max()) <= 2.0 ** -7
