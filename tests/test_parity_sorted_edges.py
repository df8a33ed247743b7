"""GPU parity of the calls around rows sorted by expert where values or sizes are at an end,
against float64.

u = 2^-24 is half a step of fp32.  A sigmoid is within 8 u of its value, and 0 may stand for
one below 2^-126."""
import numpy as np
import pytest

from tests.test_parity_block import U, Guarded, _close, _dt, _f64, _torch, _up
from tests.test_parity_sorted import _i32, _route_grad_tol
from oracle import sorted_oracle as S

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -126


# ------------------------------------------------------------------- saturated sigmoids

def _saturated():
    """Gates around the places where e^-g passes fp32's range (88.7) and where it leaves the
    correction's (104), both ends and what lies between."""
    return np.concatenate([np.linspace(-110, -80, 481), np.linspace(80, 110, 61), [0.0]])


@pytest.mark.parametrize("kind", ["channel", "token", "full"])
@pytest.mark.parametrize("gt", ["f32", "bf16"])
def test_norm_out_saturated_gates(gpu_lib, kind, gt):
    """alpha, the product with y and the sum with a residual of 0 round once each: 11 u."""
    torch = _torch()
    g = _saturated()
    T, H = (len(g), 40) if kind == "token" else (7, len(g))
    gate = _up(np.tile(g, (T, 1)) if kind == "full" else g, gt)
    y, res = _up(np.random.default_rng(0).uniform(0.5, 2.0, (T, H)), "f32"), torch.zeros(T, H, device="cuda")
    out = Guarded((T, H), "f32")
    gpu_lib.moe_norm_out(gpu_lib.make_norm(H, gate=kind, gate_act="sigmoid", alpha=0.75), y, res, gate, out.t)
    torch.cuda.synchronize()
    g = _f64(gate)
    ref = 0.75 * _f64(y) / (1.0 + np.exp(-(g[:, None] if kind == "token" else g)))
    _close(_f64(out.check()), ref, 11 * U * ref + 2 * TINY, kind)


@pytest.mark.parametrize("rows", ["few", "tile"])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("code", ["int4", "fp4"])
@pytest.mark.parametrize("group", [32, 128])
def test_q4_swiglu_saturated_gates(gpu_lib, rows, xt, code, group):
    """Matrices that pass a gate and an up value through: the sums are exact, so the error is
    the sigmoid's 8 u and that of two products, 10 u; a sigmoid taken as 0 leaves gate * up of 2^-126."""
    torch = _torch()
    rng = np.random.default_rng(0)
    K, N = 256, 10 if rows == "few" else 750
    one = 1 if code == "int4" else 2
    codes = np.zeros((2 * N, K // 2), np.uint8)
    codes[:N, 0], codes[N:, 0] = one, one << 4  # gate: input 0, up: input 1
    scales = torch.ones(2 * N, K // group, device="cuda")
    zeros = torch.zeros(2 * N, K // group, dtype=torch.uint8, device="cuda") if code == "int4" else None
    scales = torch.full_like(scales, 127, dtype=torch.uint8) if code == "fp4" and group == 32 else scales
    q4 = gpu_lib.make_q4(torch.from_numpy(codes).cuda(), scales, zeros, code=code, act="swiglu")
    g = _saturated()
    for part in [g[i:i + 16] for i in range(0, len(g), 16)] if rows == "few" else [np.tile(g, 3)]:
        x = np.zeros((len(part), K))
        x[:, 0], x[:, 1] = part, rng.uniform(-1, 1, len(part))
        x, y = _up(x, xt), Guarded((len(part), N), "f32")
        gpu_lib.moe_q4_linear(q4, x, y.t)
        torch.cuda.synchronize()
        gate, up = _f64(x)[:, :1], _f64(x)[:, 1:2]
        ref = gate / (1 + np.exp(-gate)) * up
        _close(_f64(y.check()), np.tile(ref, (1, N)), 10 * U * np.abs(ref) + 2 * TINY * np.abs(gate * up) + TINY,
               f"gates from {part[0]}")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("lt", ["bf16", "f32"])
def test_route_grad_saturated_logits(gpu_lib, renorm, lt):
    """Picked logits where 1 - s leaves fp32's range."""
    torch = _torch()
    rng = np.random.default_rng(1)
    top = _saturated()
    T, E, k = len(top), 70, 4
    lg = rng.standard_normal((T, E))
    lg[:, 3] = top
    ids = np.tile(np.array([3, 9, 40, 69]), (T, 1))
    lg = _up(lg, lt)
    s = S.scores(_f64(lg)[np.arange(T)[:, None], ids], "sigmoid")
    w = _up(s / s.sum(1, keepdims=True) if renorm else s, "f32")
    g, out = _up(rng.standard_normal((T, k)), "f32"), Guarded((T, E), "f32")
    gpu_lib.moe_route_grad(gpu_lib.make_router(E, k, scoring="sigmoid", renorm=renorm), lg, _i32(ids), w, g, out.t)
    torch.cuda.synchronize()
    args = (_f64(lg), ids, _f64(w), _f64(g), "sigmoid", renorm)
    ref, mag = S.route_grad(*args)
    far = 2 * TINY * np.abs(_f64(w)).max() * 2 * np.abs(_f64(g)).max()
    _close(_f64(out.check()), ref, _route_grad_tol(*args, ref, mag, _dt("f32")) + far, "saturated")


# ------------------------------------------------------------------- scales that are not a row's own

@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("K", [96, 160, 224, 416, 1184])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("xt,few", [("bf16", False), ("bf16", True), ("f32", False)])
def test_q4_reads_no_scale_but_a_row_s_own(gpu_lib, xt, few, grouped, K, act):
    """MXFP4, an odd number of groups a row, so that rows end inside a stage: every row's
    result is the same whatever the other rows' scales are and what lies behind the last."""
    torch = _torch()
    rng = np.random.default_rng(K)
    num, N, T = (3, 751, 1500) if grouped else (1, 1301 if act == "none" else 751, 1300)
    T = 37 if few else T
    R, G = N * (2 if act == "swiglu" else 1), K // 32
    codes = torch.from_numpy(rng.integers(0, 256, (num, R, K // 2), dtype=np.uint8)).cuda()
    good = torch.from_numpy(rng.integers(117, 126, (num, R, G), dtype=np.uint8)).cuda()
    x = _up(rng.standard_normal((T, K)) / K ** 0.5, xt)
    offsets = _i32([0, T // 2, T // 2 + 1, T])

    def product(scales):
        y = Guarded((T, N), "f32")
        q4 = gpu_lib.make_q4(codes, scales, code="fp4", act=act)
        gpu_lib.moe_q4_grouped(q4, x, offsets, y.t) if grouped else gpu_lib.moe_q4_linear(q4, x, y.t)
        return y.check()
    want = product(good)
    assert bool(want.isfinite().all())
    for byte in (255, 254, 253):
        # behind the last: a view of a longer buffer; at every place that a word's bytes can have
        for shift in range(4):
            far = torch.full((shift + good.numel() + 64,), byte, dtype=torch.uint8, device="cuda")
            view = far[shift:shift + good.numel()].view(good.shape)
            view.copy_(good)
            assert torch.equal(product(view), want), f"{byte} behind the last scale, {shift}"
        for odd in (0, 1):  # every second output's rows, gate and up alike
            other = good.clone().view(num, -1, N, G)
            other[:, :, odd::2] = byte
            got = product(other.view(good.shape))
            assert torch.equal(got[:, 1 - odd::2], want[:, 1 - odd::2]), f"{byte} in the rows between"


# ------------------------------------------------------------------- the largest sizes

@pytest.mark.parametrize("T,H", [(1 << 20, 32768 - 8), (5, 65536)])
def test_unpermute_largest(gpu_lib, T, H):
    """Up to 2^32 threads' worth of rows: few rows of ys, found from every token."""
    torch = _torch()
    M = 3
    ys = torch.randn(M, H, device="cuda").bfloat16()
    rows = (torch.arange(T, dtype=torch.int32, device="cuda") % (M + 1) - 1).view(T, 1)  # every fourth dropped
    out = torch.full((T * H + 8,), 77, dtype=torch.bfloat16, device="cuda")
    gpu_lib.moe_unpermute(ys, rows, None, None, out[:T * H].view(T, H))
    want = torch.cat([torch.zeros_like(ys[:1]), ys])
    at = out[:T * H].view(T, H)
    for t0 in range(0, T, 1 << 14):
        part = at[t0:t0 + (1 << 14)]
        assert torch.equal(part, want[torch.arange(t0, t0 + len(part), device="cuda") % (M + 1)]), t0
    assert bool((out[T * H:] == 77).all())


# ------------------------------------------------------------------- a confident router's gradient

@pytest.mark.parametrize("E,k,T", [(2, 1, 5), (8, 2, 9), (70, 1, 12), (256, 8, 40), (300, 6, 33), (1000, 8, 12),
                                   (1024, 64, 5)])
@pytest.mark.parametrize("lt", ["f32", "bf16"])
def test_route_grad_of_a_confident_router(gpu_lib, E, k, T, lt):
    """Softmax weights that are not renormalised, one expert far above the rest: its gradient
    w g (1 - s) - s (the other picks' g w) has all its digits, not those of w g alone.

    Each exponential carries |x - top| roundings of its argument and 4 more, the sum of the
    others at most E/64 + 16, quotient and result fewer than 8; the picks' part is formed in double."""
    torch = _torch()
    rng = np.random.default_rng(E + k)
    lg = rng.standard_normal((T, E))
    lead = rng.integers(0, E, T)
    gap = np.resize([0.0, 6.0, 12.0, 15.0, 18.0, 25.0, 40.0, 80.0], T)
    lg[np.arange(T), lead] = lg.max(1) + gap
    lg = _up(lg, lt)
    x = _f64(lg)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k].astype(np.int32)
    if k > 4:
        ids[T // 2, 2:4] = ids[T // 2, 0]  # the leader picked three times
        ids[T // 3, 1] = -1
    ex = np.exp(x - x.max(1, keepdims=True))
    total = ex.sum(1, keepdims=True)
    w = _up(np.take_along_axis(ex / total, np.maximum(ids, 0), 1), "f32")
    g, out = _up(rng.standard_normal((T, k)), "f32"), Guarded((T, E), "f32")
    gpu_lib.moe_route_grad(gpu_lib.make_router(E, k, scoring="softmax", renorm=False), lg, _i32(ids), w, g, out.t)
    torch.cuda.synchronize()
    gw = np.where(ids >= 0, _f64(g) * _f64(w), 0.0)
    ref, mag = np.zeros((T, E)), np.zeros((T, E))
    for t, e in np.ndindex(T, E):
        mine = ids[t] == e
        away = np.delete(ex[t], e).sum() / total[t, 0]  # 1 - s, by its own terms
        s = ex[t, e] / total[t, 0]
        ref[t, e] = gw[t, mine].sum() * away - s * gw[t, ~mine].sum()
        mag[t, e] = np.abs(gw[t, mine]).sum() * away + s * np.abs(gw[t, ~mine]).sum()
    far = (x.max(1) - x.min(1))[:, None]
    _close(_f64(out.check()), ref, (far + E / 64 + 16 + 12) * U * mag + TINY, "confident")
