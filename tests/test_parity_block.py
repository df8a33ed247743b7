"""GPU parity of the calls around the experts (norms, grouped routing, many
requests' adapters) against the float64 oracle, through the C ABI.

Tolerances count roundings.  u = 2^-24 is half a step of fp32 relative to the
value, half(t) half a step of the output's type (bf16 2^-8, fp32 2^-24).

norm_in: an element is x rs w with rs common to its row.  The sum of squares
rounds at most H/64 + 8 times in a row (64 partial sums at least, then a tree),
rs carries half of that, and division, root and products fewer than 8 more:
c(H) = H/64 + 16 roundings, relative to the element.

norm_out: r = residual + alpha g z.  z carries c(H), the sigmoid's exponent |g|
roundings of its argument (exp's error grows with the argument's rounding) and
4 more: |dr| <= u ((c + 8 + |g|) |alpha g z| + 2 |r|).  next = r / sqrt(mean r^2):
|dnext| <= |w| rs |dr| + |next| (|dr|_2 / |r|_2 + c u), the middle term from the
change of the row's norm.

lora: sums of K and r terms in any grouping that adds at most K/16 + 32 (r + 8)
of them in a row: |dv| <= (K/16 + 32) u |A||x|, and v as two bf16 parts for bf16
outputs is off by at most 2^-16 |v|."""
import math

import numpy as np
import pytest

from mxfp4_routed_expert_renorm_amd import workloads as W
from oracle import block_oracle as B
from oracle import moe_oracle as O
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GUARD = 64


def _torch():
    import torch
    return torch


def _half(t):
    torch = _torch()
    return torch.finfo(t).eps / 2


def _dt(name):
    torch = _torch()
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _up(a, dtype, shift=0):
    """A device tensor of these values, `shift` elements past a 256-byte boundary."""
    torch = _torch()
    t = torch.from_numpy(np.asarray(a, np.float32).copy()).to(_dt(dtype))
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
    v = buf[shift:].view(t.shape)
    v.copy_(t)
    return v


def _f64(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """An output with untouched elements before and behind it."""

    def __init__(self, shape, dtype, shift=0, fill=None):
        torch = _torch()
        n = int(np.prod(shape))
        dtype = torch.int32 if dtype == "i32" else _dt(dtype)
        self.buf = torch.full((n + 2 * GUARD + shift,), 77, dtype=dtype, device="cuda")
        self.t = self.buf[GUARD + shift:GUARD + shift + n].view(shape)
        self.lo, self.hi = GUARD + shift, GUARD + shift + n
        if fill is not None:
            self.t.copy_(fill)

    def check(self):
        assert bool((self.buf[:self.lo] == 77).all()) and bool((self.buf[self.hi:] == 77).all()), "wrote outside"
        return self.t


def _close(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), what
    ok = np.isfinite(ref)
    over = np.abs(got - ref)[ok] - np.broadcast_to(tol, ref.shape)[ok]
    worst = float(over.max()) if over.size else 0.0
    assert worst <= 0, f"{what}: over the tolerance by {worst:.3e}"


def _c(H):
    return H / 64 + 16


# ------------------------------------------------------------------------ norms

HS = [1, 2, 7, 63, 64, 65, 255, 256, 257, 1000, 2047, 2048, 4096, 4100, 5000, 8192, 8200, 16383, 16384]


@pytest.mark.parametrize("H", HS)
@pytest.mark.parametrize("xt,wt,ot", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("f32", "bf16", "bf16"),
                                      ("bf16", "f32", "f32")])
def test_norm_in(gpu_lib, H, xt, wt, ot):
    torch = _torch()
    T = 5 if H > 4096 else 11
    rng = np.random.default_rng(H)
    for shift, offset, weight in ((0, 0.0, True), (1, 1.0, True), (3, 0.0, False)):
        x = _up(rng.standard_normal((T, H)) * np.exp(rng.standard_normal(H)), xt, shift)
        w = _up(rng.standard_normal(H) * 0.3 + 1, wt, shift) if weight else None
        out = Guarded((T, H), ot, shift)
        gpu_lib.moe_norm_in(gpu_lib.make_norm(H, 1e-6, pre=w, weight_offset=offset), x, out.t)
        torch.cuda.synchronize()
        ref = B.rms(_f64(x), None if w is None else _f64(w), float(np.float32(1e-6)), offset)
        _close(_f64(out.check()), ref, np.abs(ref) * (_c(H) * U + _half(_dt(ot))), f"norm_in H={H} shift={shift}")


GATES = [("none", "none"), ("channel", "none"), ("token", "sigmoid"), ("full", "sigmoid"), ("full", "none"),
         ("channel", "sigmoid")]


def _norm_out_ref(y, res, gate, post_w, pre_w, kind, act, alpha, post, offset, eps, rt, nt):
    """(out, its tolerance, next, its tolerance) from float64 inputs."""
    T, H = y.shape
    r = B.norm_out(y, res, post_w, eps, gate, kind, act, alpha, post, offset)
    g = B.gate_factor(gate, kind, act, T, H)
    raw = B.gate_factor(gate, kind, "none", T, H) if act == "sigmoid" else np.zeros((T, H))
    part = np.abs(r - res)
    dr = U * ((_c(H) + 8 + np.abs(raw)) * part + 2 * np.abs(r) + 1e-30)
    nxt = B.rms(r, pre_w, eps, offset)
    rs = 1 / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    w = np.ones(H) if pre_w is None else offset + pre_w
    rel = np.linalg.norm(dr, axis=1, keepdims=True) / np.maximum(np.linalg.norm(r, axis=1, keepdims=True), 1e-300)
    dn = np.abs(w) * rs * dr + np.abs(nxt) * (rel + _c(H) * U)
    del g
    return r, dr + np.abs(r) * _half(rt), nxt, dn + np.abs(nxt) * _half(nt)


@pytest.mark.parametrize("H", [1, 63, 256, 1000, 2047, 4096, 5001, 8192, 16384])
@pytest.mark.parametrize("kind,act", GATES)
def test_norm_out(gpu_lib, H, kind, act):
    torch = _torch()
    rng = np.random.default_rng(H + len(kind))
    T, eps = 5, float(np.float32(1e-5))
    combos = [("bf16", "bf16", "bf16", "bf16", "bf16", True), ("f32", "f32", "f32", "f32", "f32", True),
              ("bf16", "f32", "f32", "bf16", "bf16", False), ("f32", "bf16", "bf16", "f32", "f32", True),
              ("bf16", "f32", "bf16", "f32", "bf16", True)]
    for n, (yt, rt, gt, wt, nt, post) in enumerate(combos):
        shift, offset, alpha = n % 3, float(n % 2), [1.0, 0.25, -2.0][n % 3]
        y, res = _up(rng.standard_normal((T, H)), yt, shift), _up(rng.standard_normal((T, H)) * 2, rt, shift)
        gshape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[kind]
        gate = None if gshape is None else _up(rng.standard_normal(gshape) * 2, gt, shift)
        pw, qw = _up(rng.standard_normal(H), wt, shift), (_up(rng.standard_normal(H), wt) if n % 2 else None)
        norm = gpu_lib.make_norm(H, 1e-5, post=pw, post_norm=post, weight_offset=offset, gate=kind, gate_act=act,
                                 alpha=alpha)
        nxt = gpu_lib.make_norm(H, 1e-5, pre=qw, weight_offset=offset)
        out, nout = Guarded((T, H), rt, shift), Guarded((T, H), nt, shift)
        gpu_lib.moe_norm_out(norm, y, res, gate, out.t, nxt, nout.t)
        alone = Guarded((T, H), rt, shift)
        gpu_lib.moe_norm_out(norm, y, res, gate, alone.t)
        torch.cuda.synchronize()
        ref, tol, nref, ntol = _norm_out_ref(_f64(y), _f64(res), None if gate is None else _f64(gate), _f64(pw),
                                             None if qw is None else _f64(qw), kind, act, alpha, post, offset, eps,
                                             _dt(rt), _dt(nt))
        _close(_f64(out.check()), ref, tol, f"out {n}")
        _close(_f64(nout.check()), nref, ntol, f"next {n}")
        assert torch.equal(alone.check(), out.t), "out differs without the next norm"


def test_norm_rows_are_independent_and_nonfinite_rows_stay_alone(gpu_lib):
    """A row of zeros norms to zeros, a row with an infinity or NaN spoils no other."""
    torch = _torch()
    H, T = 1000, 6
    rng = np.random.default_rng(1)
    x = rng.standard_normal((T, H)).astype(np.float32)
    clean = _up(x, "bf16")
    x[1], x[2, 5], x[4, 999] = 0.0, np.nan, np.inf
    bad, a, b = _up(x, "bf16"), Guarded((T, H), "f32"), Guarded((T, H), "f32")
    norm = gpu_lib.make_norm(H)
    gpu_lib.moe_norm_in(norm, clean, a.t)
    gpu_lib.moe_norm_in(norm, bad, b.t)
    torch.cuda.synchronize()
    a, b = a.check(), b.check()
    for t in (0, 3, 5):
        assert torch.equal(a[t], b[t])
    assert bool((b[1] == 0).all()) and bool(b[2].isnan().all()) and bool(b[4, 999].isnan())


def test_norm_eps_zero_and_tiny_rows(gpu_lib):
    torch = _torch()
    x = _up(np.array([[1e-15, -1e-15, 1e-15, 1e-15], [3e4, 3e4, -3e4, 3e4]]), "f32")
    out = Guarded((2, 4), "f32")
    gpu_lib.moe_norm_in(gpu_lib.make_norm(4, 0.0), x, out.t)
    torch.cuda.synchronize()
    _close(_f64(out.check()), np.sign(_f64(x)), 32 * U, "unit rows")


@pytest.mark.parametrize("H", [255, 4096])
def test_norm_in_place(gpu_lib, H):
    """out over x, over the residual, over y; next_out over y: the same bits."""
    torch = _torch()
    rng = np.random.default_rng(2)
    T = 9
    y, res = _up(rng.standard_normal((T, H)), "bf16"), _up(rng.standard_normal((T, H)), "bf16")
    w = _up(rng.standard_normal(H), "bf16")
    n = gpu_lib.make_norm(H, pre=w, post=w)
    want, nwant = torch.empty_like(y), torch.empty_like(y)
    gpu_lib.moe_norm_out(n, y, res, None, want, n, nwant)
    for out_over, next_over in (("res", None), ("y", None), ("res", "y"), ("y", "res")):
        b = {"y": y.clone(), "res": res.clone()}
        out = b[out_over]
        nout = torch.empty_like(y) if next_over is None else b[next_over]
        gpu_lib.moe_norm_out(n, b["y"], b["res"], None, out, n, nout)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(nout, nwant), (out_over, next_over)
    same, x = torch.empty_like(y), y.clone()
    gpu_lib.moe_norm_in(n, y, same)
    gpu_lib.moe_norm_in(n, x, x)
    torch.cuda.synchronize()
    assert torch.equal(x, same)


def test_norm_many_rows(gpu_lib):
    """More rows than a launch of few workgroups would cover, each with its own answer."""
    torch = _torch()
    T, H = 70001, 96
    x = torch.randn(T, H, device="cuda")
    out = Guarded((T, H), "f32")
    gpu_lib.moe_norm_in(gpu_lib.make_norm(H), x, out.t)
    ref = x.double() / (x.double().square().mean(1, keepdim=True) + float(np.float32(1e-6))).sqrt()
    assert float(((out.check().double() - ref).abs() / ref.abs().clamp_min(1e-30)).max()) <= _c(H) * U + U


@pytest.mark.parametrize("T,H", [(20001, 96), (2501, 2047), (1100, 4096), (300, 16383)])
@pytest.mark.parametrize("kind,act", [("none", "none"), ("channel", "sigmoid"), ("token", "none"), ("full", "none")])
def test_norm_out_more_rows_than_the_chip_holds(gpu_lib, T, H, kind, act):
    """Workgroups that take several rows, the last turn ragged: every row against
    float64, a broken row alone, in place, without the next norm or the post norm."""
    torch = _torch()
    rng = np.random.default_rng(T)
    eps = float(np.float32(1e-5))
    y, res = _up(rng.standard_normal((T, H)), "bf16", 1), _up(rng.standard_normal((T, H)) * 2, "bf16")
    gshape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[kind]
    gate = None if gshape is None else _up(rng.standard_normal(gshape), "bf16")
    w = _up(rng.standard_normal(H), "bf16")
    for post in (True, False):
        norm = gpu_lib.make_norm(H, 1e-5, pre=w, post=w, post_norm=post, gate=kind, gate_act=act, alpha=0.5)
        out, nout, alone = Guarded((T, H), "bf16"), Guarded((T, H), "f32", 1), Guarded((T, H), "bf16")
        gpu_lib.moe_norm_out(norm, y, res, gate, out.t, norm, nout.t)
        gpu_lib.moe_norm_out(norm, y, res, gate, alone.t)
        a, b = y.clone(), res.clone()
        gpu_lib.moe_norm_out(norm, a, b, gate, b, norm, a)
        torch.cuda.synchronize()
        ref, tol, nref, ntol = _norm_out_ref(_f64(y), _f64(res), None if gate is None else _f64(gate), _f64(w), _f64(w),
                                             kind, act, 0.5, post, 0.0, eps, torch.bfloat16, torch.float32)
        _close(_f64(out.check()), ref, tol, "out")
        _close(_f64(nout.check()), nref, ntol, "next")
        assert torch.equal(alone.check(), out.t) and torch.equal(b, out.t) and torch.equal(a, nout.t.bfloat16())
        bad = y.clone()
        bad[T - 1, 3], bad[5, H - 1] = float("nan"), float("inf")
        a, b = torch.empty_like(res), torch.empty(T, H, device="cuda")
        gpu_lib.moe_norm_out(norm, bad, res, gate, a, norm, b)
        torch.cuda.synchronize()
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[[5, T - 1]] = False
        assert torch.equal(a[keep], out.t[keep]) and torch.equal(b[keep], nout.t[keep])
        assert bool(a[T - 1, 3].isnan()) and not bool(a[5, H - 1].isfinite()) and bool(b[T - 1].isnan().all())


# ---------------------------------------------------------------------- routing

def _route(gpu_lib, logits, k, bias=None, lt="f32", shift=0, **kw):
    torch = _torch()
    T = logits.shape[0]
    lg = _up(logits, lt, shift)
    b = None if bias is None else _up(bias, "f32", shift)
    ids, w = Guarded((T, k), "i32", shift), Guarded((T, k), "f32", shift)
    gpu_lib.moe_route_groups(gpu_lib.make_router(logits.shape[1], k, **kw), lg, b, ids.t, w.t)
    torch.cuda.synchronize()
    rid, rw = B.route_groups(_f64(lg), k, bias=None if b is None else _f64(b), **kw)
    got_i, got_w = ids.check().cpu().numpy(), _f64(w.check())
    assert np.array_equal(got_i, rid), (kw, np.argwhere(got_i != rid)[:4])
    # scores and their sum in at most 16 roundings of 2^-24; the last one, to fp32, is
    # off by half of 2^-149 below 2^-126, where fp32's steps stop shrinking
    _close(got_w, rw, np.abs(rw) * 16 * U + 2.0 ** -150, f"weights {kw}")
    return got_i, got_w


ROUTERS = [dict(E=1, k=1), dict(E=2, k=2), dict(E=8, k=2, groups=4, topk_groups=1),
           dict(E=63, k=63, groups=9, topk_groups=9), dict(E=64, k=6, groups=64, topk_groups=17),
           dict(E=65, k=5, groups=5, topk_groups=2), dict(E=100, k=7, groups=20, topk_groups=3),
           dict(E=256, k=8, groups=8, topk_groups=4), dict(E=256, k=8), dict(E=256, k=64, groups=4, topk_groups=1),
           dict(E=300, k=11, groups=4, topk_groups=2), dict(E=320, k=8, groups=32, topk_groups=9),
           dict(E=1000, k=8, groups=50, topk_groups=7), dict(E=1024, k=64, groups=16, topk_groups=5),
           dict(E=1024, k=1)]


@pytest.mark.parametrize("cfg", ROUTERS, ids=lambda c: "-".join(map(str, c.values())))
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_route_groups(gpu_lib, cfg, scoring):
    cfg = dict(cfg)
    E, k = cfg.pop("E"), cfg.pop("k")
    rng = np.random.default_rng(E + k)
    n = 0
    for T in (1, 3, 37):
        for gscore in ("max", "top2"):
            for lt in ("f32", "bf16"):
                n += 1
                bias = 0.1 * rng.standard_normal(E) if n % 3 else None
                _route(gpu_lib, 1.5 * rng.standard_normal((T, E)), k, bias, lt, n % 2, scoring=scoring,
                       group_score=gscore, renorm=n % 2 == 0, scale=[1.0, 2.5, -0.5][n % 3], **cfg)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("gscore", ["max", "top2"])
def test_route_groups_masks(gpu_lib, scoring, gscore):
    """Masked experts, rows with fewer live experts than picks, rows with none,
    NaN and infinite logits, biases of -inf, +inf and NaN."""
    rng = np.random.default_rng(9)
    E, k = 64, 6
    lg = rng.standard_normal((12, E))
    lg[0] = -np.inf
    lg[1] = np.nan
    lg[2, 3:] = -np.inf
    lg[3, :60] = -np.inf
    lg[4, ::2] = np.nan
    lg[5, 7] = np.inf
    lg[6, [9, 40, 41]] = np.inf
    lg[7] = np.float32(np.finfo(np.float32).min)
    lg[8] = np.inf
    lg[9, 1:] = -np.inf
    lg[10, :] = 0.0
    lg[11, 8:] = -np.inf
    bias = 0.1 * rng.standard_normal(E)
    hard = bias.copy()
    hard[[0, 5, 63]], hard[[17, 18]], hard[20] = -np.inf, np.inf, np.nan
    for b in (None, bias, hard):
        for kw in (dict(), dict(groups=8, topk_groups=2), dict(groups=32, topk_groups=3), dict(groups=64, topk_groups=6)):
            for renorm in (True, False):
                _route(gpu_lib, lg, k, b, scoring=scoring, group_score=gscore, renorm=renorm, **kw)


def test_route_groups_ties(gpu_lib):
    """Equal choices go to the lower expert and the lower group, across lanes and rounds."""
    rng = np.random.default_rng(10)
    lg = rng.integers(-2, 3, (64, 256)).astype(np.float32)
    for kw in (dict(), dict(groups=8, topk_groups=3), dict(groups=64, topk_groups=9)):
        for gscore in ("max", "top2"):
            _route(gpu_lib, lg, 12, None, "bf16", group_score=gscore, **kw)
            _route(gpu_lib, np.zeros((3, 256)), 12, np.zeros(256), group_score=gscore, scoring="softmax", **kw)


def test_route_groups_choices_closer_than_fp32(gpu_lib):
    """Scores one fp32 step of the logit apart near 1, where their fp32 images are
    equal, and scores and biases that cancel: the order of the double values."""
    E = 64
    lg = np.zeros((4, E), np.float32)
    lg[0] = np.float32(12.0) + np.arange(E) % 7 * np.float32(2.0 ** -20)
    lg[1] = np.float32(14.0) + np.arange(E)[::-1] * np.float32(2.0 ** -19)
    lg[2] = np.float32(1e-6) * (np.arange(E) % 11)
    lg[3] = np.float32(9.0) - np.arange(E) * np.float32(2.0 ** -19)
    bias = np.zeros(E, np.float32)
    for b in (None, bias, bias + np.float32(0.75)):
        for kw in (dict(), dict(groups=8, topk_groups=2)):
            _route(gpu_lib, lg, 8, b, **kw)
    one = np.float32(1 / (1 + np.exp(-lg.astype(np.float64)[3])))
    _route(gpu_lib, np.repeat(lg[3:], 2, 0), 8, -one)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [48, 256, 640])
def test_route_groups_crowds(gpu_lib, E, scoring):
    """Choices crowded into a few fp32 steps, so that fp32 scores tell neither the
    experts nor the groups apart; some rows with only a few in the crowd; biases at
    and beyond 8, where fp32 sums lose the score's bits; logits thousands apart,
    whose softmax underflows even in double precision."""
    rng = np.random.default_rng(E)
    T, k = 40, 7
    step = np.float32(2.0 ** -22)
    tight = np.float32(2.0) + rng.integers(0, 9, (T, E)).astype(np.float32) * step
    mixed = np.where(rng.random((T, E)) < 12 / E, tight, -1.0 - rng.random((T, E)).astype(np.float32))
    far = -2000.0 * rng.random((T, E)).astype(np.float32)
    plain = rng.standard_normal((T, E)).astype(np.float32)
    small = rng.integers(0, 5, E).astype(np.float32) * step
    wide = np.where(rng.random(E) < 0.3, rng.choice([8.0, -8.0, 7.9, 8.1, 1e4, -1e30], E), 0.1 * rng.standard_normal(E))
    wide = (wide + small).astype(np.float32)
    for kw in (dict(), dict(groups=8, topk_groups=3), dict(groups=16, topk_groups=9)):
        for gscore in ("max", "top2"):
            for lg in (tight, mixed, far, plain):
                for bias in (None, small, wide):
                    _route(gpu_lib, lg, k, bias, scoring=scoring, group_score=gscore, renorm=lg is not plain, **kw)


def test_route_groups_matches_moe_route(gpu_lib):
    """Softmax over one group, renormalised, is moe_route."""
    torch = _torch()
    lg = _up(W.router_logits(31, (1,), 200, 256), "f32")
    i0, i1 = (torch.empty(200, 8, dtype=torch.int32, device="cuda") for _ in range(2))
    w0, w1 = (torch.empty(200, 8, device="cuda") for _ in range(2))
    gpu_lib.moe_route(lg, 8, i0, w0)
    gpu_lib.moe_route_groups(gpu_lib.make_router(256, 8, scoring="softmax"), lg, None, i1, w1)
    torch.cuda.synchronize()
    assert torch.equal(i0, i1)
    assert float((w0 - w1).abs().max()) <= 1e-6


# --------------------------------------------------------------------- adapters

def _lora_case(gpu_lib, T, K, N, r, num, xt, yt, seed, ids=None, ranks=None, scale=True, base=True, shift=0, poison=()):
    torch = _torch()
    rng = np.random.default_rng(seed)
    x = _up(rng.standard_normal((T, K)), xt, shift)
    a = rng.standard_normal((num, r, K)) * K ** -0.5
    b = rng.standard_normal((num, N, r)) * r ** -0.5
    for i in poison:
        a[i], b[i] = np.nan, np.inf
    if ranks is not None:  # what lies behind an adapter's rank is never used
        for i, n in enumerate(ranks):
            a[i, max(0, n):], b[i, :, max(0, n):] = np.nan, np.inf
    A, Bt = _up(a, "bf16", shift), _up(b, "bf16", shift)
    sc = _up(rng.uniform(0.5, 2.0, num), "f32") if scale else None
    rk = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
    if ids is None:
        ids = rng.integers(-1, num + 1, T)
    idt = torch.tensor(np.asarray(ids), dtype=torch.int32, device="cuda")
    bs = _up(rng.standard_normal((T, N)), yt, shift) if base else None
    out = Guarded((T, N), yt, shift)
    lora = gpu_lib.make_lora(A, Bt, scale=sc, ranks=rk)
    gpu_lib.moe_lora_add(lora, x, idt, bs, out.t)
    torch.cuda.synchronize()
    ref, tx, tv = B.lora_add(_f64(x), ids, None if bs is None else _f64(bs), _f64(A), _f64(Bt),
                             None if sc is None else _f64(sc), ranks)
    split = 2.0 ** -16 if yt == "bf16" else 0.0
    tol = (K / 16 + 32) * U * tx + ((r + 8) * U + split) * tv + np.abs(ref) * (_half(_dt(yt)) + U) + 1e-30
    _close(_f64(out.check()), ref, tol, f"lora T={T} K={K} N={N} r={r} {xt} {yt}")
    if base:  # tokens without an adapter keep the base's bits
        for t in np.flatnonzero((np.asarray(ids) < 0) | (np.asarray(ids) >= num)):
            assert torch.equal(out.t[t], bs[t]), t
    return lora, x, idt, bs, out.t


TYPES = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")]


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("K,N,r", [(1, 1, 1), (7, 5, 3), (64, 64, 8), (257, 100, 9), (256, 8, 16), (1000, 513, 17),
                                   (2048, 300, 32), (4096, 256, 64), (136, 1032, 128), (2047, 65, 127)])
def test_lora(gpu_lib, K, N, r, xt, yt):
    for n, T in enumerate((1, 2, 15, 17, 70, 300)):
        _lora_case(gpu_lib, T, K, N, r, 5, xt, yt, seed=K + T, shift=n % 3, base=n % 4 != 3, scale=n % 2 == 0)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("T", [1, 16, 33, 64, 130, 515])
def test_lora_orders_ranks_and_poisoned_neighbours(gpu_lib, T, xt, yt):
    """Adapters in runs, in turn and all alike; ranks from nothing to past the
    bank's; an adapter full of NaN and infinities that none of the checked tokens
    uses, in the same batch or not at all."""
    ranks = [0, 1, 7, 16, 24, 40, -3]
    for order in ("runs", "turn", "one", "none"):
        ids = {"runs": np.arange(T) * 7 // T, "turn": np.arange(T) % 7, "one": np.full(T, 3),
               "none": np.where(np.arange(T) % 2, -1, 1 << 30)}[order]
        _lora_case(gpu_lib, T, 512, 192, 24, 7, xt, yt, seed=T, ids=ids, ranks=ranks)
        _lora_case(gpu_lib, T, 384, 96, 16, 8, xt, yt, seed=T + 1, ids=ids, poison=(7,))


@pytest.mark.parametrize("T", [5, 64, 300])
def test_lora_a_broken_adapter_touches_only_its_tokens(gpu_lib, T):
    torch = _torch()
    lora, x, ids, base, want = _lora_case(gpu_lib, T, 512, 256, 16, 4, "bf16", "bf16", seed=3, ids=np.arange(T) % 4)
    want = want.clone()
    a, b, _, _ = lora._tensors
    a[2] = float("nan")
    b[2] = float("inf")
    out = torch.empty_like(base)
    gpu_lib.moe_lora_add(lora, x, ids, base, out)
    torch.cuda.synchronize()
    mine = (ids == 2)
    assert torch.equal(out[~mine], want[~mine])
    assert not bool(out[mine].isfinite().any())
    x[1] = float("nan")  # and a broken token only itself
    gpu_lib.moe_lora_add(lora, x, ids, base, out)
    torch.cuda.synchronize()
    keep = ~mine
    keep[1] = False
    assert torch.equal(out[keep], want[keep]) and bool(out[1].isnan().all())


@pytest.mark.parametrize("T", [5, 2000])
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_lora_nan_of_any_payload_stays_nan(gpu_lib, T, yt):
    """NaN whose payload lies in the bits that bf16 does not have."""
    torch = _torch()
    lora, x, ids, base, want = _lora_case(gpu_lib, T, 512, 256, 16, 4, "f32", yt, seed=6, ids=np.arange(T) % 4)
    want = want.clone()
    x.view(torch.int32)[1, 7] = 0x7F800001
    x.view(torch.int32)[3, 500] = -1                        # 0xffffffff
    x.view(torch.int32)[4, 0] = 0x7F800001 - (1 << 31)      # 0xff800001
    out = torch.empty_like(base)
    gpu_lib.moe_lora_add(lora, x, ids, base, out)
    torch.cuda.synchronize()
    broken = torch.zeros(T, dtype=torch.bool, device="cuda")
    broken[[1, 3, 4]] = True
    assert bool(out[broken].isnan().all()) and torch.equal(out[~broken], want[~broken])


@pytest.mark.parametrize("T", [3, 80, 700])
def test_lora_in_place_and_repeatable(gpu_lib, T):
    torch = _torch()
    lora, x, ids, base, want = _lora_case(gpu_lib, T, 4096, 512, 16, 6, "bf16", "bf16", seed=4)
    for _ in range(3):
        y = base.clone()
        gpu_lib.moe_lora_add(lora, x, ids, y, y)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_lora_empty_bank_and_no_tokens(gpu_lib):
    torch = _torch()
    a = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    b = torch.empty(0, 32, 8, dtype=torch.bfloat16, device="cuda")
    lora = gpu_lib.make_lora(a, b)
    x, ids = torch.randn(20, 64, device="cuda"), torch.zeros(20, dtype=torch.int32, device="cuda")
    base = torch.randn(20, 32, device="cuda")
    out = torch.empty_like(base)
    gpu_lib.moe_lora_add(lora, x, ids, base, out)
    torch.cuda.synchronize()
    assert torch.equal(out, base)
    gpu_lib.moe_lora_add(lora, x, ids, None, out)
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    gpu_lib.moe_lora_add(lora, x[:0], ids[:0], base[:0], out[:0])
    gpu_lib.moe_norm_in(gpu_lib.make_norm(32), base[:0], out[:0])
    gpu_lib.moe_norm_out(gpu_lib.make_norm(32), base[:0], base[:0], None, out[:0])
    gpu_lib.moe_route_groups(gpu_lib.make_router(32, 2), base[:0], None, ids[:0].view(0, 1).expand(0, 2).contiguous(),
                             base[:0, :2].contiguous())
    torch.cuda.synchronize()


# ------------------------------------------------ offsets past 32 bits of elements

def test_far_rows_of_large_calls(gpu_lib):
    """Rows whose element offsets pass 2^31: the bits of a call on those rows alone."""
    torch = _torch()
    rows, H = 2000, 4096
    T = 300 * rows                                       # 2.46e9 elements
    some = torch.randn(rows, H, device="cuda").bfloat16()
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x.view(-1, rows, H).copy_(some)
    x[-rows:] = some.flip(0)
    tail = x[-rows:].clone()
    out, want = torch.empty_like(x), torch.empty_like(tail)
    norm = gpu_lib.make_norm(H, post=torch.ones(H, device="cuda"))
    gpu_lib.moe_norm_in(norm, x, out)
    gpu_lib.moe_norm_in(norm, tail, want)
    torch.cuda.synchronize()
    assert torch.equal(out[-rows:], want)
    gpu_lib.moe_norm_out(norm, x, x, None, out)
    gpu_lib.moe_norm_out(norm, tail, tail, None, want)
    torch.cuda.synchronize()
    assert torch.equal(out[-rows:], want)
    a = torch.randn(3, 16, H, device="cuda").bfloat16()
    b = torch.randn(3, H, 16, device="cuda").bfloat16()
    ids = (torch.arange(T, device="cuda") // 500 % 4).int()
    lora = gpu_lib.make_lora(a, b)
    gpu_lib.moe_lora_add(lora, x, ids, x, out)
    gpu_lib.moe_lora_add(lora, tail, ids[-rows:].clone(), tail, want)
    torch.cuda.synchronize()
    assert torch.equal(out[-rows:], want)
    del x, out
    T, E, k = 1 << 20, 1024, 8
    lg = torch.empty(T, E, device="cuda")                # 1.07e9 elements, 4.3e9 bytes
    one = torch.randn(4096, E, device="cuda")
    lg.view(-1, 4096, E).copy_(one)
    lg[-4096:] = one.flip(0)
    i0, w0 = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    i1, w1 = torch.empty(4096, k, dtype=torch.int32, device="cuda"), torch.empty(4096, k, device="cuda")
    router = gpu_lib.make_router(E, k, groups=8, topk_groups=3)
    gpu_lib.moe_route_groups(router, lg, None, i0, w0)
    gpu_lib.moe_route_groups(router, lg[-4096:].clone(), None, i1, w1)
    torch.cuda.synchronize()
    assert torch.equal(i0[-4096:], i1) and torch.equal(w0[-4096:], w1)


@pytest.mark.parametrize("T", [7, 2000])
def test_lora_far_adapters(gpu_lib, T):
    """The last adapters of a bank of 2.6e9 elements: the bits of a bank of them alone."""
    torch = _torch()
    num, r, K, N = 5000, 128, 4096, 4096
    small_a = torch.randn(2, r, K, device="cuda").bfloat16()
    small_b = torch.randn(2, N, r, device="cuda").bfloat16()
    a, b = torch.zeros(num, r, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(num, N, r, dtype=torch.bfloat16,
                                                                                    device="cuda")
    a[-2:], b[-2:] = small_a, small_b
    x = torch.randn(T, K, device="cuda").bfloat16()
    ids = (torch.arange(T, device="cuda") * 2 // T).int()
    base = torch.randn(T, N, device="cuda").bfloat16()
    out, want = torch.empty_like(base), torch.empty_like(base)
    gpu_lib.moe_lora_add(gpu_lib.make_lora(a, b), x, ids + (num - 2), base, out)
    gpu_lib.moe_lora_add(gpu_lib.make_lora(small_a, small_b), x, ids, base, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------------------------- the run of them

def _block(gpu_lib, T, E, H, I, k, seed, prefill):
    """A block's state, its calls in order, and the oracle's outputs."""
    torch = _torch()
    rng = np.random.default_rng(seed)
    num, r, eps = 4, 16, float(np.float32(1e-6))
    bank = W.fp4_bank(seed, W.S_BANK, E, H, I)
    res = _up(rng.standard_normal((T, H)), "bf16")
    pre, post, nxt = (_up(1 + 0.1 * rng.standard_normal(H), "bf16") for _ in range(3))
    wr = _up(rng.standard_normal((E, H)) * H ** -0.5, "f32")
    bias = _up(0.02 * rng.standard_normal(E), "f32")
    gate = _up(rng.standard_normal(T), "f32")
    ids = torch.tensor(rng.integers(-1, num, T), dtype=torch.int32, device="cuda")
    mk = lambda n, m: (_up(rng.standard_normal((num, r, m)) * m ** -0.5, "bf16"),  # noqa: E731
                       _up(rng.standard_normal((num, n, r)) * 0.2, "bf16"))
    ra, la = mk(E, H), mk(H, H)
    d_bank = torch.from_numpy(bank).cuda()
    layer = gpu_lib.make_layer(H, I, fp4_base=d_bank, fp4_stride=bank.shape[1], num_slots=E)
    norm = gpu_lib.make_norm(H, 1e-6, pre=pre, post=post, gate="token", gate_act="sigmoid", alpha=0.5)
    after = gpu_lib.make_norm(H, 1e-6, pre=nxt)
    router = gpu_lib.make_router(E, k, groups=4, topk_groups=2, scale=1.5)
    rl, ll = gpu_lib.make_lora(*ra), gpu_lib.make_lora(*la)
    e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    xn, lg, pid, pw = e(T, H), e(T, E, t=torch.float32), e(T, k, t=torch.int32), e(T, k, t=torch.float32)
    y, out, xnext = e(T, H), e(T, H), e(T, H)
    if prefill:
        ws = torch.empty(gpu_lib.moe_prefill_workspace_bytes(H, I, T, k, False), dtype=torch.uint8, device="cuda")
    else:
        ws = gpu_lib.expert_workspace(H, I, T, k, False)

    def step():
        gpu_lib.moe_norm_in(norm, res, xn)
        gpu_lib.moe_router_logits(xn, wr, lg)
        gpu_lib.moe_lora_add(rl, xn, ids, lg, lg)
        gpu_lib.moe_route_groups(router, lg, bias, pid, pw)
        if prefill:
            gpu_lib.moe_prefill_forward(layer, xn, k, pid, pw, y, ws)
        else:
            gpu_lib.moe_expert_forward(layer, xn, T, k, pid, None, pw, y, ws)
        gpu_lib.moe_lora_add(ll, xn, ids, y, y)
        gpu_lib.moe_norm_out(norm, y, res, gate, out, after, xnext)

    def check():
        """Each step against the oracle on the step's own inputs."""
        x64 = _f64(xn)
        ref = B.rms(_f64(res), _f64(pre), eps)
        _close(x64, ref, np.abs(ref) * (_c(H) * U + 2.0 ** -8), "norm_in")
        hid = ids.cpu().numpy()
        plain = x64 @ _f64(wr).T
        ref, tx, tv = B.lora_add(x64, hid, plain, _f64(ra[0]), _f64(ra[1]))
        mag = np.abs(x64) @ np.abs(_f64(wr)).T
        _close(_f64(lg), ref, (H / 16 + 32) * U * (tx + mag) + (r + 8) * U * tv + 4 * U * np.abs(ref), "logits")
        rid, rw = B.route_groups(_f64(lg), k, bias=_f64(bias), groups=4, topk_groups=2, scale=1.5)
        assert np.array_equal(pid.cpu().numpy(), rid)
        _close(_f64(pw), rw, rw * 16 * U, "weights")
        fwd = O.prefill_forward if prefill else O.layer_forward
        ym = fwd(x64, rid, rw, lambda i: bank[i], H, I)
        yref, _, _ = B.lora_add(x64, hid, ym, _f64(la[0]), _f64(la[1]))
        # the experts' own tolerance (normwise 2e-2), then one more rounding
        _close(_f64(y), yref, (2e-2 + 2.0 ** -7) * np.abs(yref).max(), "block output")
        ref, tol, nref, ntol = _norm_out_ref(_f64(y), _f64(res), _f64(gate), _f64(post), _f64(nxt), "token", "sigmoid",
                                             0.5, True, 0.0, eps, torch.bfloat16, torch.bfloat16)
        _close(_f64(out), ref, tol, "stream")
        _close(_f64(xnext), nref, ntol, "next block's input")
    keep = (d_bank, ra, la, pre, post, nxt)
    return step, check, (xn, lg, pid, pw, y, out, xnext), keep


@pytest.mark.parametrize("T,prefill", [(1, False), (5, False), (40, True)])
def test_block_run(gpu_lib, T, prefill):
    step, check, _, _ = _block(gpu_lib, T, 16, 512, 256, 4, 100 + T, prefill)
    step()
    _torch().cuda.synchronize()
    check()
    log(f"block run T={T} prefill={prefill} ok")


def test_block_run_captured_and_on_another_stream(gpu_lib):
    """The run captured into a graph and replayed between eager runs, and made on a
    side stream: the eager bits each time."""
    torch = _torch()
    step, check, outs, _ = _block(gpu_lib, 40, 16, 512, 256, 4, 77, True)
    step()
    torch.cuda.synchronize()
    check()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    torch.cuda.synchronize()
    for rep in range(4):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), rep
        if rep % 2:
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for o in outs:
        o.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_two_graphs_and_two_streams_share_descriptors(gpu_lib):
    """Two graphs of calls with the same descriptors, replayed on two streams at
    once: nothing between the calls is shared."""
    torch = _torch()
    rng = np.random.default_rng(8)
    H, E, k, T = 1024, 64, 6, 50
    norm, router = gpu_lib.make_norm(H), gpu_lib.make_router(E, k, groups=8, topk_groups=3)
    a, b = _up(rng.standard_normal((3, 8, H)) * 0.03, "bf16"), _up(rng.standard_normal((3, E, 8)), "bf16")
    lora = gpu_lib.make_lora(a, b)
    ids = torch.tensor(rng.integers(0, 3, T), dtype=torch.int32, device="cuda")
    sets = []
    for i in range(2):
        x = _up(rng.standard_normal((T, H)), "bf16")
        s = dict(x=x, n=torch.empty_like(x), lg=torch.empty(T, E, device="cuda"),
                 i=torch.empty(T, k, dtype=torch.int32, device="cuda"), w=torch.empty(T, k, device="cuda"))
        sets.append(s)

    def go(s):
        gpu_lib.moe_norm_in(norm, s["x"], s["n"])
        gpu_lib.moe_lora_add(lora, s["n"], ids, None, s["lg"])
        gpu_lib.moe_route_groups(router, s["lg"], None, s["i"], s["w"])
    want = []
    for s in sets:
        go(s)
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in s.items()})
    streams, graphs = [torch.cuda.Stream() for _ in sets], []
    for st, s in zip(streams, sets):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            go(s)
        graphs.append(g)
    torch.cuda.synchronize()
    for rep in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            assert all(torch.equal(s[n], w[n]) for n in s), rep


def test_binding_refuses_bad_tensors(gpu_lib):
    torch = _torch()
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="dense"):
        gpu_lib.moe_norm_in(gpu_lib.make_norm(32), x[:, ::2], torch.zeros(4, 32, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        gpu_lib.moe_norm_in(gpu_lib.make_norm(64), x, torch.zeros(3, 64, device="cuda"))
    with pytest.raises(TypeError):
        gpu_lib.moe_norm_in(gpu_lib.make_norm(64), x.half(), x)
    with pytest.raises(ValueError, match="device"):
        gpu_lib.moe_norm_in(gpu_lib.make_norm(64, pre=torch.ones(64)), x, torch.empty_like(x))
    with pytest.raises(ValueError, match="gate"):
        gpu_lib.moe_norm_out(gpu_lib.make_norm(64, gate="token"), x, x, None, torch.empty_like(x))
    with pytest.raises(TypeError):
        gpu_lib.moe_norm_out(gpu_lib.make_norm(64), x, x, None, x.bfloat16())
    with pytest.raises(ValueError, match="shape"):
        gpu_lib.moe_route_groups(gpu_lib.make_router(32, 2), x, None, torch.zeros(4, 2, dtype=torch.int32, device="cuda"),
                                 torch.zeros(4, 2, device="cuda"))
    with pytest.raises(TypeError):
        gpu_lib.moe_route_groups(gpu_lib.make_router(64, 2), x, None, torch.zeros(4, 2, dtype=torch.int64, device="cuda"),
                                 torch.zeros(4, 2, device="cuda"))
    with pytest.raises(gpu_lib.MoeError, match="next_out"):
        gpu_lib.moe_norm_out(gpu_lib.make_norm(64), x, x, None, x, gpu_lib.make_norm(64), x)
    assert math.isfinite(float(x.sum()))


def _call_under_test(B, torch, call):
    """The call's tensors by name and a function that makes the call with them."""
    def new(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    if call == "route":
        r = B.make_router(64, 2)
        t = {"logits": new(4, 64), "bias": new(64), "ids": new(4, 2, dtype=torch.int32), "w": new(4, 2)}
        return t, lambda t: B.moe_route_groups(r, t["logits"], t["bias"], t["ids"], t["w"])
    if call == "norm_in":
        n = B.make_norm(64)
        return {"x": new(4, 64), "out": new(4, 64)}, lambda t: B.moe_norm_in(n, t["x"], t["out"])
    if call == "lora":
        lora = B.make_lora(new(2, 4, 64, dtype=torch.bfloat16), new(2, 32, 4, dtype=torch.bfloat16))
        t = {"x": new(4, 64), "ids": new(4, dtype=torch.int32), "base": new(4, 32), "out": new(4, 32)}
        return t, lambda t: B.moe_lora_add(lora, t["x"], t["ids"], t["base"], t["out"])
    n = B.make_norm(64, gate=call)
    t = {"y": new(4, 64), "residual": new(4, 64), "gate": new(*{"channel": (64,), "token": (4,), "full": (4, 64)}[call]),
         "out": new(4, 64), "next_out": new(4, 64)}
    return t, lambda t: B.moe_norm_out(n, t["y"], t["residual"], t["gate"], t["out"], n, t["next_out"])


@pytest.mark.parametrize("call", ["route", "norm_in", "channel", "token", "full", "lora"])
def test_binding_refuses_each_wrong_tensor(gpu_lib, call):
    torch = _torch()
    good, run = _call_under_test(gpu_lib, torch, call)
    run(good)
    for name, t in good.items():
        wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device="cuda")
        for bad, error in ((t.to(torch.float16), TypeError), (t.to(torch.int64), TypeError),
                           (torch.cat([t, t]), ValueError), (t[None], ValueError), (wide, ValueError),
                           (wide[..., ::2], ValueError), (t.cpu(), ValueError)):
            with pytest.raises(error):
                run({**good, name: bad})
    torch.cuda.synchronize()
    run(good)
