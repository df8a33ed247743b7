"""GPU parity of moe_lora_add's two forms, each at the sizes, types and values
where it can go wrong, against the float64 oracle.

Tolerances count roundings, u = 2^-24 half a step of fp32, half(t) half a step of
the output's type.  v = scale A x is an fp32 sum of K terms, at most K/16 + 32 of
them added in a row: |dv| <= (K/16 + 32) u |A||x|.  The matrix units take v as
three bf16 parts whose sum it is, so B v adds at most 3 r + 8 products in a row:
(3 r + 8) u |B||v|.  The sum with the base rounds once to fp32, once to the
output's type."""
import os
import re

import numpy as np
import pytest

from oracle import block_oracle as B
from tests.test_parity_block import TYPES, U, Guarded, _close, _dt, _f64, _half, _torch, _up

pytestmark = pytest.mark.gpu

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_routed_expert_renorm_amd",
                      "csrc", "lora.hip")


def _token_form(T, K, N, r):
    """The library's choice of the form (test_the_rule_is_the_librarys holds the two together)."""
    return T <= 128 or (T * r * (K + N) <= 24e6 and (T <= 512 or (r <= 16 and T <= 1536)))


def _lora(gpu_lib, T, K, N, r, num, xt, yt, seed, ids=None, base=True, scale=True, shift=0):
    torch = _torch()
    rng = np.random.default_rng(seed)
    x = _up(rng.standard_normal((T, K)), xt, shift)
    a, b = _up(rng.standard_normal((num, r, K)) * K ** -0.5, "bf16", shift), _up(
        rng.standard_normal((num, N, r)) * r ** -0.5, "bf16", shift)
    sc = _up(rng.uniform(0.5, 2.0, num), "f32") if scale else None
    if ids is None:
        ids = np.sort(rng.integers(-1, num + 1, T))
    bs = _up(rng.standard_normal((T, N)), yt, shift) if base else None
    out = Guarded((T, N), yt, shift)
    gpu_lib.moe_lora_add(gpu_lib.make_lora(a, b, scale=sc), x, torch.tensor(ids, dtype=torch.int32, device="cuda"), bs,
                         out.t)
    torch.cuda.synchronize()
    ref, tx, tv = B.lora_add(_f64(x), ids, None if bs is None else _f64(bs), _f64(a), _f64(b),
                             None if sc is None else _f64(sc))
    tol = (K / 16 + 32) * U * tx + (3 * r + 8) * U * tv + np.abs(ref) * (_half(_dt(yt)) + U) + 1e-30
    _close(_f64(out.check()), ref, tol, f"lora T={T} K={K} N={N} r={r} {xt} {yt}")


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("T", [40, 1601])
def test_lora_sums_keep_24_bits(gpu_lib, T, xt, yt):
    """v of 24 significant bits under a base that cancels its upper ones: what is
    left is the lower bits, exactly."""
    torch = _torch()
    num, N = 50, 70
    rng = np.random.default_rng(T)
    scale = (1 + rng.integers(0, 1 << 23, num) * 2.0 ** -23).astype(np.float32) * np.float32(2.0) ** rng.integers(
        -9, 9, num).astype(np.float32)
    scale[:3] = np.array([0x3F80FFFF, 0x3F817FFF, 0x3FFFFFFF], np.uint32).view(np.float32)
    sc = _up(scale, "f32")
    x = _up(np.ones((T, 8)), xt)
    a, b = torch.zeros(num, 1, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(num, N, 1, dtype=torch.bfloat16,
                                                                                 device="cuda")
    a[:, :, 0] = 1.0
    ids = torch.arange(T, dtype=torch.int32, device="cuda") % num
    mine = sc[ids.long()]
    base = (-mine.bfloat16()).to(_dt(yt))[:, None].expand(T, N).contiguous()
    out = Guarded((T, N), yt)
    gpu_lib.moe_lora_add(gpu_lib.make_lora(a, b, scale=sc), x, ids, base, out.t)
    torch.cuda.synchronize()
    want = (mine.double()[:, None] + base.double()).to(_dt(yt))
    assert torch.equal(out.check(), want), float((out.t.double() - want.double()).abs().max())


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [37, 1603])
def test_lora_without_an_adapter_keeps_the_bases_bits(gpu_lib, T, yt):
    """-0, NaN of any payload, infinities and subnormals of the base, beside tokens
    that have adapters: for ids outside the bank and for adapters of rank 0."""
    torch = _torch()
    K, N, r, num = 64, 200, 24, 3
    rng = np.random.default_rng(T)
    x = _up(rng.standard_normal((T, K)), "bf16")
    a, b = _up(rng.standard_normal((num, r, K)), "bf16"), _up(rng.standard_normal((num, N, r)), "bf16")
    ranks = torch.tensor([24, 0, 7], dtype=torch.int32, device="cuda")
    bits = torch.int32 if yt == "f32" else torch.int16
    base = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (T, N))).to("cuda").to(bits)  # any pattern at all
    base[:, ::5] = torch.iinfo(bits).min  # -0
    base = base.view(_dt(yt))
    for ids in (torch.arange(T) % 4, torch.full((T,), -1), torch.full((T,), 1), torch.arange(T) * 5 // T - 1):
        ids = ids.to("cuda", torch.int32)
        out = Guarded((T, N), yt)
        gpu_lib.moe_lora_add(gpu_lib.make_lora(a, b, ranks=ranks), x, ids, base, out.t)
        torch.cuda.synchronize()
        alone = (ids < 0) | (ids >= num) | (ids == 1)
        assert torch.equal(out.check()[alone].view(bits), base[alone].view(bits))


def test_the_rule_is_the_librarys():
    with open(SOURCE) as f:
        body = re.search(r"bool token_form\(.*?\n}", f.read(), re.S).group(0)
    assert "(double)T * L->r * ((double)L->K + L->N)" in body
    assert "T <= 128 || (products <= 24e6 && (T <= 512 || (L->r <= 16 && T <= 1536)))" in body


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("K", [1, 7, 63, 65, 200])
@pytest.mark.parametrize("N", [1, 7, 8, 63, 71, 130])
def test_lora_tiles_of_small_and_odd_sizes(gpu_lib, K, N, xt, yt):
    """The tile form without a whole slab of K or a whole block of outputs, with
    ranks whose last pieces run into the next rows, with and without base and scale."""
    for n, r in enumerate((1, 3, 9, 17, 40)):
        T = 1537 + 23 * n
        assert not _token_form(T, K, N, r)
        _lora(gpu_lib, T, K, N, r, 5, xt, yt, seed=K + N + r, base=(n + K) % 2 == 0, scale=(n + N) % 3 != 0, shift=n % 3)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("base", [True, False])
def test_lora_tiles_of_many_adapters(gpu_lib, xt, yt, base):
    """Every token of a tile with an adapter of its own, in runs, in turn: one to 16
    adapters a tile, one to 64 steps, with ranks 8 to 128, with and without a base."""
    for r, num, T in ((8, 40, 1601), (33, 20, 1540), (128, 17, 529)):
        assert not _token_form(T, 192, 256, r)
        for ids in (np.arange(T) % (num + 1), np.arange(T) * num // T, np.arange(T) // 5 % num):
            _lora(gpu_lib, T, 192, 256, r, num, xt, yt, seed=r, ids=ids, base=base)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("T,K,N,r", [(3, 65536, 40, 8), (3, 40, 65536, 8), (5, 8200, 4104, 48), (513, 65536, 24, 8),
                                     (513, 24, 65536, 8), (1537, 5000, 4100, 16), (530, 4104, 6001, 72)])
def test_lora_long_inputs_and_outputs(gpu_lib, T, K, N, r, xt, yt):
    """K or N above 4096, up to the largest that is taken, in both forms."""
    assert _token_form(T, K, N, r) == (T < 128)
    _lora(gpu_lib, T, K, N, r, 3, xt, yt, seed=T + K, base=r != 8 or T < 100, scale=True, shift=T % 2)
