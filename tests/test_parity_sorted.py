"""GPU parity of the rows' way to the experts and back, with the gradients, against the
float64 oracle.

Tolerances count roundings, u = 2^-24 half a step of fp32, half(t) half a step of the
output's type.  unpermute: a term's product and its way through at most k + 1 sums are
k + 2 roundings of the terms' magnitudes.  gw: a thread adds H/64 + 8 products in a row at
most, then a tree of fewer than 16.  gys: one product.  route_grad: the sigmoid within
8 roundings, the difference from the mean (formed in double) one, products and the
repeated picks' sums fewer than k + 4; a softmax's exponential carries |x - top|
roundings of its argument, sums of at most E/64 + 16 terms in a row and 8 more."""
import numpy as np
import pytest

from oracle import block_oracle as BO
from oracle import sorted_oracle as S
from tests.test_parity_block import U, Guarded, _close, _dt, _f64, _half, _torch, _up

pytestmark = pytest.mark.gpu


def _i32(a):
    return _torch().from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _ids(rng, T, k, E, dropped):
    """Distinct picks where E allows, skewed; some outside [0, E)."""
    p = np.exp(rng.standard_normal(E))
    if k <= E:
        ids = np.argsort(-(np.log(p / p.sum()) + rng.gumbel(size=(T, E))), axis=1)[:, :k]
    else:
        ids = rng.integers(0, E, (T, k))
    bad = rng.choice([-1, -7, E, 2 ** 31 - 1, -2 ** 31], (T, k))
    return np.where(rng.random((T, k)) < dropped, bad, ids).astype(np.int32)


def _scratch(lib, T, k, E, fill=0xA5):
    n = lib.moe_permute_scratch_bytes(T, k, E)
    return _torch().full((n,), fill, dtype=_torch().uint8, device="cuda") if n else None


def _permute(lib, x, ids, E, scratch="new", stream=None):
    """(xs or None, offsets, perm, rows), guarded."""
    T, k = ids.shape
    out = [Guarded((E + 1,), "i32"), Guarded((max(T * k, 1),), "i32"), Guarded((T, k), "i32")]
    xs = None
    if x is not None:
        xs = Guarded((T * k, x.shape[1]), {2: "bf16", 4: "f32"}[x.element_size()], 1)
    lib.moe_permute(x, ids, None if xs is None else xs.t, out[0].t, out[1].t[:T * k], out[2].t,
                    _scratch(lib, T, k, E) if isinstance(scratch, str) else scratch, stream=stream)
    return xs, *out


def _check_permute(x, ids, E, got):
    torch = _torch()
    xs, offsets, perm, rows = got
    o, p, r = S.sort_pairs(ids, E)
    assert np.array_equal(offsets.check().cpu().numpy(), o)
    assert np.array_equal(rows.check().cpu().numpy(), r)
    gp = perm.check().cpu().numpy()
    assert np.array_equal(gp[:len(p)], p) and (gp[len(p):] == 77).all(), "perm, or what is behind its end"
    if xs is not None:
        t = xs.check()
        want = x[torch.from_numpy(p // ids.shape[1]).long().cuda()]
        bits = torch.int16 if x.element_size() == 2 else torch.int32
        assert torch.equal(t[:len(p)].view(bits), want.view(bits))
        assert bool((t[len(p):] == 77).all()), "rows behind the last expert's"


@pytest.mark.parametrize("T,k,E,H", [
    (1, 1, 1, 1), (1, 8, 256, 4096), (2, 3, 5, 7), (3, 64, 8, 65), (7, 6, 300, 2047), (64, 8, 256, 512), (63, 4, 1, 33),
    (128, 8, 64, 100), (255, 8, 1024, 8), (300, 12, 17, 257), (511, 8, 256, 24), (512, 8, 256, 24), (513, 8, 250, 24),
    (777, 6, 300, 129), (1000, 9, 1000, 16), (1200, 7, 40, 515), (1025, 8, 256, 1030), (4096, 8, 256, 40),
    (5000, 13, 1023, 9), (3, 2, 9, 65536)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_permute(gpu_lib, T, k, E, H, xt):
    rng = np.random.default_rng(T + k + E)
    for dropped in (0.0, 0.3):
        ids = _ids(rng, T, k, E, dropped)
        x = _up(rng.standard_normal((T, H)), xt, 1)
        _check_permute(x, ids, E, _permute(gpu_lib, x, _i32(ids), E))
    _check_permute(None, ids, E, _permute(gpu_lib, None, _i32(ids), E))


@pytest.mark.parametrize("T,k,E", [(5, 4, 16), (600, 8, 64), (2000, 8, 256)])
def test_permute_one_expert_takes_all_or_none(gpu_lib, T, k, E):
    x = _torch().randn(T, 33, device="cuda")
    for fill in (0, E - 1, -1, E):
        ids = np.full((T, k), fill, np.int32)
        _check_permute(x, ids, E, _permute(gpu_lib, x, _i32(ids), E))


def test_permute_nothing(gpu_lib):
    torch = _torch()
    offsets = Guarded((9,), "i32")
    e = lambda *s, t=torch.int32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    gpu_lib.moe_permute(e(0, 16, t=torch.float32), e(0, 4), e(0, 16, t=torch.float32), offsets.t, e(0), e(0, 4),
                        _scratch(gpu_lib, 0, 4, 8))
    assert bool((offsets.check() == 0).all())


def test_permute_copies_bits(gpu_lib):
    """NaNs of any payload, infinities and subnormals, aligned and at row ends."""
    torch = _torch()
    rng = np.random.default_rng(5)
    for bits, dtype in ((np.int16, torch.bfloat16), (np.int32, torch.float32)):
        info = np.iinfo(bits)
        x = torch.from_numpy(rng.integers(info.min, info.max, (40, 77), dtype=bits)).cuda().view(dtype)
        ids = _ids(rng, 40, 3, 8, 0.1)
        _check_permute(x, ids, 8, _permute(gpu_lib, x, _i32(ids), 8))


def test_permute_far_rows(gpu_lib):
    """More than 2^31 elements sorted: the last rows against the first tokens'."""
    torch = _torch()
    T, k, H, E = 4200, 8, 65536, 16
    x = torch.randn(T, H, device="cuda").bfloat16()
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    xs = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    offsets, perm, rows = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    rows = rows.view(T, k)
    gpu_lib.moe_permute(x, ids, xs, offsets, perm, rows, _scratch(gpu_lib, T, k, E))
    assert torch.equal(perm.long(), ids.view(-1).sort(stable=True).indices)
    for i in list(range(0, T * k, 1531)) + [T * k - 1]:
        assert torch.equal(xs[i], x[int(perm[i]) // k]), i
    out, gw = torch.empty(T, H, device="cuda"), torch.empty(T, k, device="cuda")
    gpu_lib.moe_unpermute(xs, rows, None, None, out)
    gpu_lib.moe_unpermute_grad(out, xs, rows, None, xs, gw)
    for t in (0, T // 2, T - 1):
        assert torch.equal(out[t], x[t].float() * k)
        ref = (out[t].double() * x[t].double()).sum()
        assert float((gw[t].double() - ref).abs().max()) <= (H / 64 + 24) * U * float(ref)
        for r in (0, k - 1):
            assert torch.equal(xs[rows[t, r]], out[t].bfloat16())


SHAPES = [(1, 1, 1), (1, 8, 4096), (2, 3, 7), (5, 64, 65), (9, 9, 512), (64, 8, 520), (33, 6, 2047), (17, 12, 1000),
          (3, 8, 8200), (700, 2, 64), (130, 8, 1024), (2, 5, 65536)]


@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("yt,ot", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_unpermute(gpu_lib, T, k, H, yt, ot):
    torch = _torch()
    rng = np.random.default_rng(T + k + H)
    for n, (weighted, based) in enumerate([(True, True), (False, False), (True, False), (False, True)]):
        E = 16
        rows = S.sort_pairs(_ids(rng, T, k, E, 0.2 * (n % 2)), E)[2]
        M = T * k
        ys = rng.standard_normal((M, H))
        unread = np.setdiff1d(np.arange(M), rows)
        ys[unread] = np.nan  # rows that no pair has
        ys = _up(ys, yt, n)
        w = _up(rng.standard_normal((T, k)), "f32", n) if weighted else None
        if weighted:
            w[torch.from_numpy(rows).cuda() < 0] = float("nan")  # dropped pairs' weights
        base = _up(rng.standard_normal((T, H)), ot, n) if based else None
        out = Guarded((T, H), ot, n)
        gpu_lib.moe_unpermute(ys, _i32(rows), w, base, out.t)
        torch.cuda.synchronize()
        ref, mag = S.unpermute(_f64(ys), rows, None if w is None else _f64(w), None if base is None else _f64(base))
        _close(_f64(out.check()), ref, (k + 2) * U * mag + _half(_dt(ot)) * np.abs(ref) + 1e-40, f"unpermute {n}")
        if based:
            inplace = Guarded((T, H), ot, n, fill=base)
            gpu_lib.moe_unpermute(ys, _i32(rows), w, inplace.t, inplace.t)
            assert torch.equal(inplace.check(), out.t)


@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("gt,yt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_unpermute_grad(gpu_lib, T, k, H, gt, yt):
    torch = _torch()
    rng = np.random.default_rng(T + k + H + 1)
    for n, weighted in enumerate([True, False]):
        E = 16
        rows = S.sort_pairs(_ids(rng, T, k, E, 0.2 * n), E)[2]
        M = T * k
        ys = rng.standard_normal((M, H))
        ys[np.setdiff1d(np.arange(M), rows)] = np.nan
        ys, g = _up(ys, yt, n), _up(rng.standard_normal((T, H)), gt, 1)
        w = _up(rng.standard_normal((T, k)), "f32") if weighted else None
        gys, gw = Guarded((M, H), yt, n), Guarded((T, k), "f32", n)
        gpu_lib.moe_unpermute_grad(g, ys, _i32(rows), w, gys.t, gw.t)
        torch.cuda.synchronize()
        ref, rw, mag = S.unpermute_grad(_f64(g), _f64(ys), rows, None if w is None else _f64(w), np.full((M, H), 77.0))
        _close(_f64(gys.check()), ref, (U + _half(_dt(yt))) * np.abs(ref), "gys")
        _close(_f64(gw.check()), rw, (H / 64 + 24) * U * mag + 1e-40, "gw")
        alone, walone = Guarded((M, H), yt, n), Guarded((T, k), "f32", n)
        gpu_lib.moe_unpermute_grad(g, None, _i32(rows), w, alone.t, None)
        gpu_lib.moe_unpermute_grad(g, ys, _i32(rows), w, None, walone.t)
        inplace = ys.clone()
        wp = torch.empty_like(gw.t)
        gpu_lib.moe_unpermute_grad(g, inplace, _i32(rows), w, inplace, wp)
        live = torch.from_numpy(np.unique(rows[rows >= 0])).long().cuda()
        assert torch.equal(alone.check(), gys.t) and torch.equal(walone.check(), gw.t) and torch.equal(wp, gw.t)
        assert torch.equal(inplace[live], gys.t[live])


def test_rows_outside_and_no_rows(gpu_lib):
    """Rows past ys are dropped; without any row of ys the base, or zeros, is what comes back."""
    torch = _torch()
    ys, base = torch.randn(4, 32, device="cuda"), torch.randn(3, 32, device="cuda")
    rows = _i32([[0, 4], [-5, 2 ** 31 - 1], [-2 ** 31, 3]])
    out, gw = Guarded((3, 32), "f32"), Guarded((3, 2), "f32")
    gpu_lib.moe_unpermute(ys, rows, None, base, out.t)
    assert torch.equal(out.check(), torch.stack([base[0] + ys[0], base[1], base[2] + ys[3]]))
    gys = Guarded((4, 32), "f32")
    gpu_lib.moe_unpermute_grad(base, ys, rows, None, gys.t, gw.t)
    want = torch.full_like(ys, 77)
    want[0], want[3] = base[0], base[2]
    assert torch.equal(gys.check(), want) and bool((gw.check()[[0, 1, 1, 2], [1, 0, 1, 0]] == 0).all())
    none = ys[:0]
    gpu_lib.moe_unpermute(none, rows, None, None, out.t)
    assert bool((out.check() == 0).all())
    gpu_lib.moe_unpermute(none, rows, None, base, out.t)
    assert torch.equal(out.check(), base)
    gpu_lib.moe_unpermute_grad(base, none, rows, None, none, gw.t)
    assert bool((gw.check() == 0).all())


@pytest.mark.parametrize("T,k,H", [(6, 4, 600), (5, 3, 40)])
def test_a_nonfinite_row_stays_with_its_token(gpu_lib, T, k, H):
    torch = _torch()
    rng = np.random.default_rng(3)
    rows = _i32(S.sort_pairs(_ids(rng, T, k, 8, 0.0), 8)[2])
    ys, g, w = (_up(rng.standard_normal(s), "f32") for s in ((T * k, H), (T, H), (T, k)))
    call = lambda y, gg, ww: (gpu_lib.moe_unpermute(y, rows, ww, None, torch.empty(T, H, device="cuda")),  # noqa: E731
                              *gpu_lib.moe_unpermute_grad(gg, y, rows, ww, torch.empty_like(y),
                                                          torch.empty(T, k, device="cuda")))
    a = call(ys, g, w)
    y2, g2, w2 = ys.clone(), g.clone(), w.clone()
    y2[rows[1, 2], 5], g2[2, H - 1], w2[3, 0] = float("nan"), float("inf"), float("nan")
    b = call(y2, g2, w2)
    keep = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(a[0][keep], b[0][keep]) and bool(b[0][3].isnan().all()) and bool(b[0][1, 5].isnan())
    at = rows[[t for t in range(T) if t not in (2, 3)]].view(-1).long()
    assert torch.equal(a[1][at], b[1][at])
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(a[2][keep], b[2][keep]) and bool(b[2][1, 2].isnan())
    assert torch.equal(a[2][1, [0, 1]], b[2][1, [0, 1]])


# --------------------------------------------------------------- the router's gradient

def _route_grad_tol(lg, ids, w, g, scoring, renorm, ref, mag, ot):
    T, E = lg.shape
    k = ids.shape[1]
    tol = (8 + k + 5) * U * mag
    if scoring == "softmax" and not renorm:
        s = S.scores(lg, scoring)
        top = np.nanmax(np.where(np.isfinite(lg), lg, -np.inf), axis=1, keepdims=True)
        far = np.where(s > 0, np.abs(np.where(np.isfinite(lg), lg, 0) - np.where(np.isfinite(top), top, 0)), 0)
        tol = tol + (far + E / 64 + 24) * U * mag
    return tol + _half(ot) * np.abs(ref) + 1e-40


def _route_grad(lib, lg, ids, w, g, lt, ot, shift, **kw):
    torch = _torch()
    T, E = lg.shape
    k = ids.shape[1]
    out = Guarded((T, E), ot, shift)
    d = _up(lg, lt, shift)
    wd, gd = _up(w, "f32", shift), _up(g, "f32", shift)
    lib.moe_route_grad(lib.make_router(E, k, **kw), d, _i32(ids), wd, gd, out.t)
    torch.cuda.synchronize()
    scoring, renorm = kw.get("scoring", "sigmoid"), kw.get("renorm", True)
    args = (_f64(d), ids, _f64(wd), _f64(gd), scoring, renorm)
    ref, mag = S.route_grad(*args)
    _close(_f64(out.check()), ref, _route_grad_tol(*args, ref, mag, _dt(ot)), f"route_grad {kw}")
    return out.t


@pytest.mark.parametrize("E,k,T", [(1, 1, 1), (2, 2, 3), (7, 3, 5), (64, 6, 9), (65, 64, 4), (256, 8, 70), (257, 9, 5),
                                   (300, 6, 77), (512, 12, 6), (513, 4, 5), (1000, 8, 3), (1024, 64, 5)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad(gpu_lib, E, k, T, scoring, renorm):
    rng = np.random.default_rng(E + k)
    for n, (lt, ot) in enumerate([("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")]):
        lg = _f64(_up(3 * rng.standard_normal((T, E)), lt))
        scale = [1.0, 2.5, -0.5, 1.0][n]
        ids, w = BO.route_groups(lg, k, scoring=scoring, renorm=renorm, scale=scale)
        g = rng.standard_normal((T, k)) + (100.0 if n == 1 else 0.0)  # a part common to all picks
        _route_grad(gpu_lib, lg, ids, w, g, lt, ot, n, scoring=scoring, renorm=renorm, scale=scale)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_masks_infinities_and_repeated_picks(gpu_lib, scoring, renorm):
    rng = np.random.default_rng(4)
    T, E, k = 9, 70, 5
    lg = rng.standard_normal((T, E))
    lg[0] = -np.inf
    lg[1] = np.nan
    lg[2, ::2], lg[2, 1::4] = np.nan, -np.inf
    lg[3, 60:] = float(np.finfo(np.float32).min)
    lg[4, [3, 9]] = np.inf
    lg[5, 1:] = -np.inf
    lg[6, :] = np.linspace(-80, 80, E)
    ids, w = BO.route_groups(lg, k, scoring=scoring, renorm=renorm)
    g = rng.standard_normal((T, k))
    g[w == 0] = np.nan  # masked picks: their gradient counts for nothing
    ids[7], w[7] = [4, 4, 9, 4, 9], [0.1, 0.2, 0.3, 0.2, 0.2]
    ids[8, :2] = [-1, E]
    out = _route_grad(gpu_lib, lg, ids, w, g, "f32", "f32", 0, scoring=scoring, renorm=renorm)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_against_differences(gpu_lib, scoring, renorm):
    """The library's own weights, differences of them in double's place: a step of 2^-6 in the
    logits, whose third-order rest is below 2^-12 of the largest slope."""
    torch = _torch()
    T, E, k = 4, 24, 4
    rng = np.random.default_rng(6)
    lg = _up(rng.standard_normal((T, E)), "f32")
    g = _up(rng.standard_normal((T, k)), "f32")
    router = gpu_lib.make_router(E, k, scoring=scoring, renorm=renorm, scale=2.0)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    gpu_lib.moe_route_groups(router, lg, None, ids, w)
    out = torch.empty(T, E, device="cuda")
    gpu_lib.moe_route_grad(router, lg, ids, w, g, out)
    ids_h, g_h, h = ids.cpu().numpy(), _f64(g), 2.0 ** -6

    def loss(x):
        s = np.take_along_axis(S.scores(x, scoring), ids_h, 1)
        return (2.0 * g_h * (s / s.sum(1, keepdims=True) if renorm else s)).sum(1)
    base, num = _f64(lg), np.zeros((T, E))
    for e in range(E):
        d = np.zeros(E)
        d[e] = h
        num[:, e] = (loss(base + d) - loss(base - d)) / (2 * h)
    assert np.abs(_f64(out) - num).max() <= 2.0 ** -12 * 2 * np.abs(g_h).max() * 4


def test_route_grad_no_tokens(gpu_lib):
    torch = _torch()
    e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    gpu_lib.moe_route_grad(gpu_lib.make_router(8, 2), e(0, 8), e(0, 2, t=torch.int32), e(0, 2), e(0, 2), e(0, 8))
