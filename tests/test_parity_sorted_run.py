"""The calls around rows sorted by expert run together on the GPU, forward and back,
captured, replayed and on several streams, and what the binding refuses."""
import numpy as np
import pytest

from oracle import sorted_oracle as S
from tests.test_parity_block import _f64, _torch, _up
from tests.test_parity_q4 import Weights
from tests.test_parity_sorted import _i32, _scratch

pytestmark = pytest.mark.gpu


class Layer:
    """A sparse layer's tensors: T tokens of H, k of E experts of width I."""

    def __init__(self, lib, seed, T, E, k, H, I, dt, code, scoring="sigmoid"):
        torch = _torch()
        rng = np.random.default_rng(seed)
        self.lib, self.E, self.scoring = lib, E, scoring
        self.up = Weights(lib, rng, E, I, H, 32, code, "e8m0" if code == "fp4" else "bf16", code == "int4", "swiglu")
        self.down = Weights(lib, rng, E, H, I, 32, code, "e8m0" if code == "fp4" else "bf16", code == "int4", "none")
        self.router = lib.make_router(E, k, scoring=scoring)
        self.x, self.shared, self.g = (_up(rng.standard_normal((T, H)), dt) for _ in range(3))
        self.logits = _up(rng.standard_normal((T, E)), "f32")
        e = lambda *s, t=torch.int32: torch.full(s, 77, dtype=t, device="cuda")  # noqa: E731
        d, f = self.x.dtype, torch.float32
        self.ids, self.w, self.offsets, self.perm, self.rows = e(T, k), e(T, k, t=f), e(E + 1), e(T * k), e(T, k)
        self.xs, self.h, self.ys, self.out = e(T * k, H, t=d), e(T * k, I, t=d), e(T * k, H, t=d), e(T, H, t=d)
        self.gys, self.gw, self.gl, self.gx = e(T * k, H, t=d), e(T, k, t=f), e(T, E, t=f), e(T, H, t=d)
        self.scratch = _scratch(lib, T, k, E)

    def outputs(self):
        return [self.ids, self.w, self.offsets, self.perm, self.rows, self.xs, self.h, self.ys, self.out, self.gys,
                self.gw, self.gl, self.gx]

    def clear(self):
        for t in self.outputs():
            t.fill_(77)

    def run(self, stream=None):
        lib, s = self.lib, dict(stream=stream)
        lib.moe_route_groups(self.router, self.logits, None, self.ids, self.w, **s)
        lib.moe_permute(self.x, self.ids, self.xs, self.offsets, self.perm, self.rows, self.scratch, **s)
        lib.moe_q4_grouped(self.up.q4, self.xs, self.offsets, self.h, **s)
        lib.moe_q4_grouped(self.down.q4, self.h, self.offsets, self.ys, **s)
        lib.moe_unpermute(self.ys, self.rows, self.w, self.shared, self.out, **s)
        lib.moe_unpermute_grad(self.g, self.ys, self.rows, self.w, self.gys, self.gw, **s)
        lib.moe_route_grad(self.router, self.logits, self.ids, self.w, self.gw, self.gl, **s)
        lib.moe_unpermute(self.gys, self.rows, None, None, self.gx, **s)  # permute's gradient


def _norm_close(got, ref, rel, what):
    assert np.linalg.norm(got - ref) <= rel * np.linalg.norm(ref), what


# a product of 256 inputs passes 2 (32 + 3 * 8 + 16) roundings of 2^-24, on magnitudes some
# sqrt(256) times its value, three such steps: under 6e-4.  bf16 rounds each of the tensors
# on the way, by at most 2^-8, again three: under 2^-6
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (37, 12, 3), (300, 64, 6), (1100, 16, 6)])
@pytest.mark.parametrize("dt,rel", [("f32", 6e-4), ("bf16", 2.0 ** -6)])
@pytest.mark.parametrize("code,scoring", [("fp4", "sigmoid"), ("int4", "softmax")])
def test_a_sparse_layer_and_its_gradient(gpu_lib, T, E, k, dt, rel, code, scoring):
    torch = _torch()
    a = Layer(gpu_lib, T, T, E, k, 256, 96, dt, code, scoring)
    a.run()
    torch.cuda.synchronize()
    ids, w, x, g = a.ids.cpu().numpy(), _f64(a.w), _f64(a.x), _f64(a.g)
    offsets, perm, rows = S.sort_pairs(ids, E)
    ys = np.zeros((T * k, 256))
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        if offsets[e] < offsets[e + 1]:
            h = S.q4_product(x[perm[at] // k], a.up.matrix(e), "swiglu", 1)[0]
            ys[at] = S.q4_product(h, a.down.matrix(e), "none", 1)[0]
    _norm_close(_f64(a.ys), ys, rel, "the experts' rows")
    _norm_close(_f64(a.out), S.unpermute(ys, rows, w, _f64(a.shared))[0], rel, "out")
    gys, gw, _ = S.unpermute_grad(g, ys, rows, w, np.zeros_like(ys))
    _norm_close(_f64(a.gys), gys, rel, "gys")
    # gw are products of 256 with values that are small beside their terms: to their terms' size
    assert np.abs(_f64(a.gw) - gw).max() <= rel * np.linalg.norm(g, axis=1).max() * np.linalg.norm(ys, axis=1).max()
    _norm_close(_f64(a.gx), S.unpermute(_f64(a.gys), rows)[0], 2.0 ** -8 if dt == "bf16" else 1e-6, "gx")

    # the logits' gradient against differences of the weights' part of the loss, the experts' rows
    # and the picks fixed; gw as the library has it.  The rest is of third order: h^2 / 6 times at
    # most 8 times the largest slope
    got, gw, h = _f64(a.gl), _f64(a.gw), 2.0 ** -7
    lg = _f64(a.logits)

    def loss(v):
        s = np.take_along_axis(S.scores(v, scoring), ids, 1)
        return (gw * s / s.sum(1, keepdims=True)).sum(1)
    for e in range(0, E, max(1, E // 8)):
        d = np.zeros(E)
        d[e] = h
        num = (loss(lg + d) - loss(lg - d)) / (2 * h)
        assert np.abs(num - got[:, e]).max() <= 2 * h * h * np.abs(gw).max() * k + 1e-5 * np.abs(gw).max()


SIZES = [(3, 8, 2), (50, 64, 6), (900, 16, 8)]  # one launch to sort, and two; few rows, and tiles


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_run_captured_and_on_another_stream(gpu_lib, T, E, k, dt):
    torch = _torch()
    a = Layer(gpu_lib, 1, T, E, k, 256, 512, dt, "fp4")
    a.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in a.outputs()]
    a.clear()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.run(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a.outputs(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.run()
    logits, x = a.logits.clone(), a.x.clone()
    for rep in range(4):
        a.logits.copy_(logits.roll(rep, 0)), a.x.copy_(x.roll(rep, 0))
        a.clear()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in a.outputs()]
        a.clear()
        if a.scratch is not None:
            a.scratch.fill_(rep)
        a.run()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a.outputs(), got)), rep


@pytest.mark.parametrize("T,E,k", SIZES)
def test_two_graphs_on_two_streams_share_weights(gpu_lib, T, E, k):
    """The descriptors are shared, the tensors and the scratch are not."""
    torch = _torch()
    a, b = (Layer(gpu_lib, n, T, E, k, 256, 512, "bf16", "int4") for n in (2, 3))
    b.up, b.down, b.router = a.up, a.down, a.router
    want, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, layer in zip(streams, (a, b)):
        layer.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in layer.outputs()])
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            layer.run()
    for rep in range(5):
        a.clear(), b.clear()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for layer, ref in zip((a, b), want):
            assert all(torch.equal(p, q) for p, q in zip(layer.outputs(), ref)), rep


def test_a_padded_batch(gpu_lib):
    """Tokens whose picks are all dropped: they reach no expert and bring back their base."""
    torch = _torch()
    a = Layer(gpu_lib, 4, 40, 8, 2, 256, 96, "f32", "fp4")
    a.logits[30:] = float("-inf")  # every expert masked
    a.x[30:] = float("nan")
    a.run()
    a.ids[30:] = -1
    gpu_lib.moe_permute(a.x, a.ids, a.xs.fill_(77), a.offsets, a.perm.fill_(77), a.rows, a.scratch)
    for q4, src, dst in ((a.up.q4, a.xs, a.h), (a.down.q4, a.h, a.ys)):
        gpu_lib.moe_q4_grouped(q4, src, a.offsets, dst.fill_(77))
    gpu_lib.moe_unpermute(a.ys, a.rows, a.w, a.shared, a.out)
    gpu_lib.moe_unpermute_grad(a.g, a.ys, a.rows, a.w, a.gys.fill_(77), a.gw)
    torch.cuda.synchronize()
    assert int(a.offsets[-1]) == 60 and bool((a.rows[30:] == -1).all())
    assert torch.equal(a.out[30:], a.shared[30:]) and bool(a.out.isfinite().all())
    for t in (a.xs, a.h, a.ys, a.gys):
        assert bool((t[60:] == 77).all())
    assert bool((a.gw[30:] == 0).all()) and bool((a.gl[30:] == 0).all())


def test_the_binding_refuses(gpu_lib):
    """Each tensor of each call in a wrong type, a wrong shape, a stride, or off the GPU."""
    torch = _torch()
    a = Layer(gpu_lib, 5, 6, 8, 2, 64, 32, "f32", "fp4")
    a.run()
    few = torch.zeros(4, dtype=torch.uint8, device="cuda")
    calls = [(gpu_lib.moe_permute, [a.x, a.ids, a.xs, a.offsets, a.perm, a.rows, few], []),
             (gpu_lib.moe_unpermute, [a.ys, a.rows, a.w, a.shared, a.out], []),
             (gpu_lib.moe_unpermute_grad, [a.g, a.ys, a.rows, a.w, a.gys, a.gw], []),
             (gpu_lib.moe_route_grad, [a.logits, a.ids, a.w, a.gw, a.gl], [a.router]),
             (gpu_lib.moe_q4_grouped, [a.xs, a.offsets, a.h], [a.up.q4]),
             (gpu_lib.moe_q4_linear, [a.xs, a.h], [a.up.q4])]
    for call, args, first in calls:
        call(*first, *args)
        for i, t in enumerate(args):
            wrong = [t.cpu(), t.repeat_interleave(2, dim=0)[::2]]
            if t is not few:
                wrong += [t.to(torch.float16), t.unsqueeze(0), t[:-1] if t.numel() > 1 else t]
            for bad in wrong:
                if call is gpu_lib.moe_permute and (t is a.offsets and bad.shape == a.offsets[:-1].shape):
                    continue  # a valid call of one expert fewer
                if call is gpu_lib.moe_unpermute and bad.shape == a.ys[:-1].shape and t is a.ys:
                    continue  # fewer rows: the pairs of the others are dropped
                with pytest.raises((TypeError, ValueError)):
                    call(*first, *args[:i], bad, *args[i + 1:])
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError):
        gpu_lib.moe_unpermute(a.ys, a.rows, a.w, None, a.ys[:6])  # over an input
    with pytest.raises(RuntimeError):  # many pairs without scratch
        ids = _i32(np.zeros((5000, 2)))
        gpu_lib.moe_permute(None, ids, None, a.offsets, torch.empty_like(ids).view(-1), torch.empty_like(ids))
