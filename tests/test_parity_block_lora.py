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
