"""GPU parity of moe_lora_add's two forms, each at the sizes, types and values
where it can go wrong, against float64."""
import numpy as np
import pytest

from tests.test_parity_block import TYPES, Guarded, _dt, _torch, _up

pytestmark = pytest.mark.gpu


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
