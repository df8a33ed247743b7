"""Refusals of the calls around the experts (no GPU): the C entry points check
every argument before they touch a device, and the binding checks its tensors."""
import ctypes
import math
import os

import pytest

from mxfp4_routed_expert_renorm_amd import binding as B

FAKE, FAKE2, FAKE3 = (ctypes.c_void_p(v) for v in (0x1000, 0x2000, 0x4000))
ODD = ctypes.c_void_p(0x1001)
EINVAL, ESHAPE = 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("library not built: run __graft_entry__.build()")
    return B.load()


def _st(lib, fn, *args):
    return getattr(lib, fn)(*args), lib.moe_last_error().decode()


@pytest.mark.parametrize("name", ["moe_router", "moe_norm", "moe_lora"])
def test_binding_structs_match_header(name):
    from tests.test_abi import _struct_fields
    assert [f for f, _ in getattr(B, name)._fields_] == _struct_fields(name)


@pytest.mark.parametrize("change,status,word", [
    (dict(E=0), ESHAPE, "E=0"), (dict(E=1025), ESHAPE, "E=1025"), (dict(k=0), EINVAL, "k=0"),
    (dict(k=65, topk_groups=8), EINVAL, "k=65"), (dict(scoring=2), EINVAL, "scoring=2"),
    (dict(groups=0), EINVAL, "groups=0"), (dict(groups=7), EINVAL, "divide"), (dict(groups=128), EINVAL, "groups=128"),
    (dict(topk_groups=0), EINVAL, "topk_groups=0"), (dict(topk_groups=9), EINVAL, "topk_groups=9"),
    (dict(k=33, topk_groups=1), EINVAL, "fewer than k=33"), (dict(group_score=5), EINVAL, "group_score=5"),
    (dict(renorm=2), EINVAL, "renorm=2"), (dict(scale=math.inf), EINVAL, "scale"),
    (dict(scale=math.nan), EINVAL, "scale")])
def test_router_settings(lib, change, status, word):
    r = B.make_router(256, 8, groups=8, topk_groups=4)
    for f, v in change.items():
        setattr(r, f, v)
    st, msg = _st(lib, "moe_route_groups", ctypes.byref(r), FAKE, 0, None, 4, FAKE, FAKE, None)
    assert st == status and word in msg


def test_route_groups_arguments(lib):
    r = B.make_router(256, 8)
    call = lambda logits=FAKE, lt=0, bias=None, T=4, ids=FAKE, w=FAKE: _st(  # noqa: E731
        lib, "moe_route_groups", ctypes.byref(r), logits, lt, bias, T, ids, w, None)
    assert call(T=0, logits=None)[0] == 0
    assert call(T=-1)[0] == ESHAPE and call(T=(1 << 20) + 1)[0] == ESHAPE
    assert call(lt=2)[0] == EINVAL
    for bad in (dict(logits=None), dict(ids=None), dict(w=None), dict(logits=ODD), dict(bias=ODD), dict(ids=ODD),
                dict(w=ODD), dict(logits=ODD, lt=1)):
        assert call(**bad)[0] == EINVAL, bad
    assert _st(lib, "moe_route_groups", None, FAKE, 0, None, 4, FAKE, FAKE, None)[0] == EINVAL


def _norm(**change):
    n = B.make_norm(64)
    for f, v in change.items():
        setattr(n, f, v)
    return n


@pytest.mark.parametrize("change,status", [
    (dict(H=0), ESHAPE), (dict(H=16385), ESHAPE), (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL),
    (dict(alpha=math.inf), EINVAL), (dict(weight_offset=math.nan), EINVAL), (dict(wt=3), EINVAL),
    (dict(pre_w=0x1002), EINVAL), (dict(post_w=0x1001, wt=1), EINVAL), (dict(post_norm=2), EINVAL),
    (dict(gate=4), EINVAL), (dict(gate=-1), EINVAL), (dict(gate_act=2), EINVAL)])
def test_norm_settings(lib, change, status):
    n, good = _norm(**change), _norm()
    st, _ = _st(lib, "moe_norm_in", ctypes.byref(n), FAKE, 0, 2, FAKE2, 0, None)
    assert st == status
    st, _ = _st(lib, "moe_norm_out", ctypes.byref(n), FAKE, 0, FAKE2, None, 0, 2, FAKE3, 0, None, None, 0, None)
    assert st == status
    st, _ = _st(lib, "moe_norm_out", ctypes.byref(good), FAKE, 0, FAKE2, None, 0, 2, FAKE2, 0, ctypes.byref(n), FAKE3, 0,
                None)
    assert st == status


def test_norm_arguments(lib):
    n = _norm()
    call = lambda x=FAKE, xt=0, T=2, out=FAKE2, ot=0: _st(  # noqa: E731
        lib, "moe_norm_in", ctypes.byref(n), x, xt, T, out, ot, None)
    assert call(T=0, x=None)[0] == 0
    for bad, status in ((dict(T=-1), ESHAPE), (dict(T=(1 << 20) + 1), ESHAPE), (dict(xt=5), EINVAL), (dict(ot=-1), EINVAL),
                        (dict(x=None), EINVAL), (dict(out=None), EINVAL), (dict(x=ODD), EINVAL), (dict(out=ODD), EINVAL),
                        (dict(out=FAKE, ot=1), EINVAL)):
        assert call(**bad)[0] == status, bad
    gated, other = _norm(gate=1), _norm(H=65)
    ref = ctypes.byref

    def out(norm=n, y=FAKE, yt=0, res=FAKE2, gate=None, gt=0, T=2, out=FAKE3, rt=0, nxt=None, nout=None, nt=0):
        return _st(lib, "moe_norm_out", ref(norm), y, yt, res, gate, gt, T, out, rt, None if nxt is None else ref(nxt),
                   nout, nt, None)
    far = ctypes.c_void_p(0x8000)
    assert out(T=0, y=None)[0] == 0
    for bad, status in ((dict(T=-1), ESHAPE), (dict(y=None), EINVAL), (dict(res=None), EINVAL), (dict(out=None), EINVAL),
                        (dict(yt=2), EINVAL), (dict(rt=2), EINVAL), (dict(norm=gated), EINVAL),
                        (dict(norm=gated, gate=far, gt=7), EINVAL), (dict(gate=far), EINVAL), (dict(nxt=n), EINVAL),
                        (dict(nout=far), EINVAL), (dict(nxt=other, nout=far), ESHAPE),
                        (dict(nxt=n, nout=far, nt=9), EINVAL), (dict(nxt=n, nout=FAKE3), EINVAL),
                        (dict(out=FAKE, yt=1), EINVAL), (dict(nxt=n, nout=FAKE, nt=1), EINVAL),
                        (dict(nxt=n, nout=FAKE2, nt=1), EINVAL), (dict(norm=gated, gate=FAKE3), EINVAL),
                        (dict(norm=gated, gate=ODD), EINVAL), (dict(res=ODD), EINVAL)):
        assert out(**bad)[0] == status, bad


@pytest.mark.parametrize("change,status", [
    (dict(K=0), ESHAPE), (dict(K=65537), ESHAPE), (dict(N=0), ESHAPE), (dict(N=65537), ESHAPE), (dict(r=0), ESHAPE),
    (dict(r=129), ESHAPE), (dict(num=-1), ESHAPE), (dict(num=65537), ESHAPE), (dict(a=None), EINVAL),
    (dict(b=None), EINVAL), (dict(a=0x1001), EINVAL), (dict(scale=0x1002), EINVAL), (dict(ranks=0x1002), EINVAL)])
def test_lora_settings(lib, change, status):
    m = B.moe_lora(64, 64, 8, 4, 0x1000, 0x2000, None, None)
    for f, v in change.items():
        setattr(m, f, v)
    assert _st(lib, "moe_lora_add", ctypes.byref(m), FAKE, 1, 2, FAKE, None, FAKE2, 1, None)[0] == status


def test_lora_arguments(lib):
    m = B.moe_lora(64, 64, 8, 4, 0x1000, 0x2000, None, None)
    call = lambda x=FAKE, xt=1, T=2, ids=FAKE, base=None, out=FAKE2, yt=1: _st(  # noqa: E731
        lib, "moe_lora_add", ctypes.byref(m), x, xt, T, ids, base, out, yt, None)
    assert call(T=0, x=None)[0] == 0
    for bad, status in ((dict(T=-1), ESHAPE), (dict(T=(1 << 20) + 1), ESHAPE), (dict(x=None), EINVAL),
                        (dict(ids=None), EINVAL), (dict(out=None), EINVAL), (dict(xt=2), EINVAL), (dict(yt=4), EINVAL),
                        (dict(ids=ctypes.c_void_p(0x1002)), EINVAL), (dict(base=ODD), EINVAL), (dict(out=FAKE), EINVAL)):
        assert call(**bad)[0] == status, bad


def test_binding_refuses_tensors_off_the_gpu_and_bad_descriptors():
    import torch
    x, out = torch.zeros(2, 8), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_norm_in(B.make_norm(8), x, out)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_norm_out(B.make_norm(8), x, x, None, out)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_route_groups(B.make_router(8, 2), x, None, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))
    bank = torch.zeros(3, 2, 8, dtype=torch.bfloat16)
    up = torch.zeros(3, 4, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_lora_add(B.make_lora(bank, up), x, torch.zeros(2, dtype=torch.int32), None, torch.zeros(2, 4))
    with pytest.raises(ValueError, match="shape"):
        B.make_norm(8, pre=torch.ones(9))
    with pytest.raises(TypeError):
        B.make_norm(8, pre=torch.ones(8, dtype=torch.float16))
    with pytest.raises(TypeError):
        B.make_norm(8, pre=torch.ones(8), post=torch.ones(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dense"):
        B.make_norm(8, pre=torch.ones(16)[::2])
    with pytest.raises(ValueError):
        B.make_lora(bank, torch.zeros(2, 4, 2, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dense"):
        B.make_lora(bank.transpose(1, 2).contiguous().transpose(1, 2), up)
    with pytest.raises(TypeError):
        B.make_lora(bank.float(), up)
    with pytest.raises(TypeError):
        B.make_lora(bank, up, ranks=torch.zeros(3))
    with pytest.raises(KeyError):
        B.make_router(8, 2, scoring="relu")
