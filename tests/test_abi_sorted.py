"""Refusals of the calls around rows sorted by expert and of the products with 4-bit
weights (no GPU): invented addresses, so every call here is refused or has nothing to do."""
import ctypes

import pytest

from mxfp4_routed_expert_renorm_amd import binding as B
from tests.test_abi_block import EINVAL, ESHAPE, ODD, _st, lib  # noqa: F401
from tests.test_abi_block_overlaps import FAR, _p, _shifts

ENOMEM = 4
A = [_p(v) for v in FAR]


@pytest.mark.parametrize("name", ["moe_q4"])
def test_binding_structs_match_header(name):
    from tests.test_abi import _struct_fields
    assert [f for f, _ in getattr(B, name)._fields_] == _struct_fields(name)


def _permute(lib, x=A[0], xt=0, T=4, k=2, H=64, E=8, ids=A[1], xs=A[2], offsets=A[3], perm=A[4], rows=A[5], scratch=A[6],
             n=1 << 19):
    return _st(lib, "moe_permute", x, xt, T, k, H, E, ids, xs, offsets, perm, rows, scratch, n, None)


def test_permute_arguments(lib):  # noqa: F811
    for bad, status in ((dict(k=0), EINVAL), (dict(k=65), EINVAL), (dict(T=-1), ESHAPE), (dict(T=(1 << 19) + 1), ESHAPE),
                        (dict(E=0), ESHAPE), (dict(E=1025), ESHAPE), (dict(H=0), ESHAPE), (dict(H=65537), ESHAPE),
                        (dict(x=None), EINVAL), (dict(xs=None), EINVAL), (dict(xt=2), EINVAL), (dict(ids=None), EINVAL),
                        (dict(offsets=None), EINVAL), (dict(perm=None), EINVAL), (dict(rows=None), EINVAL),
                        (dict(x=ODD), EINVAL), (dict(xs=ODD), EINVAL), (dict(ids=ODD), EINVAL), (dict(offsets=ODD), EINVAL),
                        (dict(perm=ODD), EINVAL), (dict(rows=ODD), EINVAL), (dict(scratch=ODD), EINVAL),
                        (dict(offsets=None, T=0), EINVAL)):
        assert _permute(lib, **bad)[0] == status, bad


def test_permute_scratch(lib):  # noqa: F811
    T, k, E = 4096, 8, 256
    need = B.moe_permute_scratch_bytes(T, k, E)
    assert need > 0 and B.moe_permute_scratch_bytes(T, 65, E) == 0 and B.moe_permute_scratch_bytes(1 << 20, 2, E) == 0
    far = dict(T=T, k=k, E=E, H=1, x=None, xs=None, ids=_p(1 << 30), offsets=_p(2 << 30), perm=_p(3 << 30), rows=_p(4 << 30))
    for scratch, n in ((None, 0), (None, need), (_p(5 << 30), need - 1)):
        st, msg = _permute(lib, scratch=scratch, n=n, **far)
        assert st == ENOMEM and str(need) in msg


def test_permute_overlaps(lib):  # noqa: F811
    at = dict(x=(FAR[0], 1024), ids=(FAR[1], 32), xs=(FAR[2], 2048), offsets=(FAR[3], 36), perm=(FAR[4], 32),
              rows=(FAR[5], 32))
    for which in ("xs", "offsets", "perm", "rows"):
        for other, (start, size) in at.items():
            if other != which:
                for d in _shifts(at[which][1], size) + [0]:
                    st, msg = _permute(lib, **{which: _p(start + d)})
                    assert st == EINVAL and "overlap" in msg, (which, other, d)
    T, k, E = 4096, 8, 256
    far = dict(T=T, k=k, E=E, H=1, x=None, xs=None, ids=_p(1 << 30), offsets=_p(2 << 30), perm=_p(3 << 30), rows=_p(4 << 30))
    for other in (1, 2, 3, 4):
        st, msg = _permute(lib, scratch=_p((other << 30) + 4), **far)
        assert st == EINVAL and "overlap" in msg, other


def _unpermute(lib, ys=A[0], yt=0, M=8, rows=A[1], w=A[2], base=A[3], T=4, k=2, H=64, out=A[4], ot=0):
    return _st(lib, "moe_unpermute", ys, yt, M, rows, w, base, T, k, H, out, ot, None)


SIZES = [(dict(T=-1), ESHAPE), (dict(T=(1 << 20) + 1), ESHAPE), (dict(k=0), EINVAL), (dict(k=65), EINVAL),
         (dict(H=0), ESHAPE), (dict(H=65537), ESHAPE), (dict(M=-1), ESHAPE), (dict(M=(1 << 20) + 1), ESHAPE)]


def test_unpermute_arguments(lib):  # noqa: F811
    assert _unpermute(lib, T=0, ys=None, rows=None, out=None)[0] == 0
    for bad, status in SIZES + [(dict(yt=2), EINVAL), (dict(ot=-1), EINVAL), (dict(ys=None), EINVAL),
                                (dict(rows=None), EINVAL), (dict(out=None), EINVAL), (dict(ys=ODD), EINVAL),
                                (dict(rows=ODD), EINVAL), (dict(w=ODD), EINVAL), (dict(base=ODD), EINVAL),
                                (dict(out=ODD), EINVAL)]:
        assert _unpermute(lib, **bad)[0] == status, bad


def test_unpermute_overlaps(lib):  # noqa: F811
    for other, size in ((0, 2048), (1, 32), (2, 32), (3, 1024)):
        for d in _shifts(1024, size) + ([] if other == 3 else [0]):
            st, msg = _unpermute(lib, out=_p(FAR[other] + d))
            assert st == EINVAL and "overlap" in msg, (other, d)


def _grad(lib, g=A[0], gt=0, ys=A[1], yt=0, M=8, rows=A[2], w=A[3], T=4, k=2, H=64, gys=A[4], gw=A[5]):
    return _st(lib, "moe_unpermute_grad", g, gt, ys, yt, M, rows, w, T, k, H, gys, gw, None)


def test_unpermute_grad_arguments(lib):  # noqa: F811
    assert _grad(lib, T=0, g=None)[0] == 0 and _grad(lib, gys=None, gw=None)[0] == 0
    for bad, status in SIZES + [(dict(gt=2), EINVAL), (dict(yt=2), EINVAL), (dict(g=None), EINVAL), (dict(ys=None), EINVAL),
                                (dict(rows=None), EINVAL), (dict(g=ODD), EINVAL), (dict(ys=ODD), EINVAL),
                                (dict(rows=ODD), EINVAL), (dict(w=ODD), EINVAL), (dict(gys=ODD), EINVAL),
                                (dict(gw=ODD), EINVAL)]:
        assert _grad(lib, **bad)[0] == status, bad
    sizes = (1024, 2048, 32, 32, 2048, 32)
    for which, mine in (("gys", 4), ("gw", 5)):
        for other in range(6):
            if other != mine:
                for d in _shifts(sizes[mine], sizes[other]) + ([] if (which, other) == ("gys", 1) else [0]):
                    st, msg = _grad(lib, **{which: _p(FAR[other] + d)})
                    assert st == EINVAL and "overlap" in msg, (which, other, d)


def test_route_grad_arguments(lib):  # noqa: F811
    r = B.make_router(256, 8)

    def call(router=r, lg=A[0], lt=0, T=2, ids=A[1], w=A[2], gw=A[3], out=A[4], gt=0):
        return _st(lib, "moe_route_grad", None if router is None else ctypes.byref(router), lg, lt, T, ids, w, gw, out, gt,
                   None)
    assert call(T=0, lg=None)[0] == 0
    for bad, status in ((dict(router=None), EINVAL), (dict(router=B.make_router(2000, 8)), ESHAPE),
                        (dict(router=B.make_router(8, 9)), EINVAL), (dict(T=-1), ESHAPE), (dict(T=(1 << 20) + 1), ESHAPE),
                        (dict(lt=2), EINVAL), (dict(gt=2), EINVAL), (dict(lg=None), EINVAL), (dict(ids=None), EINVAL),
                        (dict(w=None), EINVAL), (dict(gw=None), EINVAL), (dict(out=None), EINVAL), (dict(lg=ODD), EINVAL),
                        (dict(ids=ODD), EINVAL), (dict(w=ODD), EINVAL), (dict(gw=ODD), EINVAL), (dict(out=ODD), EINVAL)):
        assert call(**bad)[0] == status, bad
    for other, size in enumerate((2048, 64, 64, 64)):
        for d in _shifts(2048, size) + [0]:
            st, msg = call(out=_p(FAR[other] + d))
            assert st == EINVAL and "overlap" in msg, (other, d)


def _q4(**change):
    q = B.moe_q4(128, 16, 4, 32, B.Q4_INT4, 0, B.MOE_BF16, FAR[0], FAR[1], FAR[2], 1024, 128, 64)
    for f, v in change.items():
        setattr(q, f, v)
    return q


@pytest.mark.parametrize("change,status", [
    (dict(K=0), ESHAPE), (dict(K=48), ESHAPE), (dict(K=65568), ESHAPE), (dict(N=0), ESHAPE), (dict(N=65537), ESHAPE),
    (dict(num=0), ESHAPE), (dict(num=1025), ESHAPE), (dict(group=0), ESHAPE), (dict(group=16), ESHAPE),
    (dict(group=96), ESHAPE), (dict(group=256), ESHAPE), (dict(code=2), EINVAL), (dict(act=2), EINVAL), (dict(st=3), EINVAL),
    (dict(st=-1), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(codes=FAR[0] + 8), EINVAL),
    (dict(scales=FAR[1] + 1), EINVAL), (dict(code=B.Q4_FP4), EINVAL), (dict(code_stride=1008), EINVAL),
    (dict(code_stride=1032), EINVAL), (dict(scale_stride=126), EINVAL), (dict(scale_stride=129), EINVAL),
    (dict(zero_stride=63), EINVAL), (dict(act=1), EINVAL)])
def test_q4_settings(lib, change, status):  # noqa: F811
    q = _q4(**change)
    assert _st(lib, "moe_q4_linear", ctypes.byref(q), A[4], 0, 2, A[5], 0, None)[0] == status
    assert _st(lib, "moe_q4_grouped", ctypes.byref(q), A[4], 0, 2, A[6], A[5], 0, None)[0] == status


def test_q4_arguments(lib):  # noqa: F811
    q = ctypes.byref(_q4())
    lin = lambda q=q, x=A[4], xt=0, T=2, y=A[5], yt=0: _st(lib, "moe_q4_linear", q, x, xt, T, y, yt, None)  # noqa: E731
    grp = lambda q=q, x=A[4], xt=0, T=2, o=A[6], y=A[5], yt=0: _st(  # noqa: E731
        lib, "moe_q4_grouped", q, x, xt, T, o, y, yt, None)
    assert lin(T=0, x=None, y=None)[0] == 0 and grp(T=0, x=None, y=None)[0] == 0
    for bad, status in ((dict(q=None), EINVAL), (dict(T=-1), ESHAPE), (dict(T=(1 << 20) + 1), ESHAPE), (dict(xt=2), EINVAL),
                        (dict(yt=2), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(x=ODD), EINVAL),
                        (dict(y=ODD), EINVAL)):
        assert lin(**bad)[0] == status and grp(**bad)[0] == status, bad
    assert grp(o=None)[0] == EINVAL and grp(o=ODD)[0] == EINVAL
    size = 2 * 16 * 4
    for other, n in ((0, 4 * 1024), (1, 4 * 128), (2, 4 * 64), (4, 2 * 128 * 4)):
        for d in _shifts(size, n) + [0]:
            for call in (lin, grp):
                st, msg = call(y=_p(FAR[other] + d))
                assert st == EINVAL and "overlap" in msg, (other, d)
    for d in _shifts(size, 20) + [0]:
        assert grp(y=_p(FAR[6] + d))[0] == EINVAL


def test_binding_refuses_tensors_off_the_gpu_and_bad_descriptors():
    import torch
    i32, u8 = torch.int32, torch.uint8
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        B.moe_permute(z(2, 8), z(2, 3, dtype=i32), z(6, 8), z(5, dtype=i32), z(6, dtype=i32), z(2, 3, dtype=i32))
    with pytest.raises(ValueError, match="both"):
        B.moe_permute(z(2, 8), z(2, 3, dtype=i32), None, z(5, dtype=i32), z(6, dtype=i32), z(2, 3, dtype=i32))
    with pytest.raises(ValueError):
        B.moe_permute(None, z(6, dtype=i32), None, z(5, dtype=i32), z(6, dtype=i32), z(6, dtype=i32))
    with pytest.raises(ValueError, match="GPU"):
        B.moe_unpermute(z(6, 8), z(2, 3, dtype=i32), z(2, 3), None, z(2, 8))
    with pytest.raises(ValueError, match="GPU"):
        B.moe_unpermute_grad(z(2, 8), z(6, 8), z(2, 3, dtype=i32), z(2, 3), z(6, 8), z(2, 3))
    with pytest.raises(ValueError, match="needs ys"):
        B.moe_unpermute_grad(z(2, 8), None, z(2, 3, dtype=i32), z(2, 3), z(6, 8), z(2, 3))
    with pytest.raises(ValueError, match="gys"):
        B.moe_unpermute_grad(z(2, 8), None, z(2, 3, dtype=i32), z(2, 3), None, None)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_route_grad(B.make_router(8, 2), z(2, 8), z(2, 2, dtype=i32), z(2, 2), z(2, 2), z(2, 8))
    codes, scales = z(3, 6, 32, dtype=u8), z(3, 6, 2)
    q = B.make_q4(codes, scales)
    assert (q.K, q.N, q.num, q.group, q.code_stride, q.scale_stride) == (64, 6, 3, 32, 192, 48)
    assert B.make_q4(codes, scales, act="swiglu").N == 3 and B.make_q4(codes[0], scales[0]).num == 1
    with pytest.raises(ValueError, match="GPU"):
        B.moe_q4_linear(q, z(2, 64), z(2, 6))
    with pytest.raises(ValueError, match="GPU"):
        B.moe_q4_grouped(q, z(2, 64), z(4, dtype=i32), z(2, 6))
    for bad in (dict(codes=z(3, 6, 32)), dict(scales=z(3, 6, 2, dtype=torch.float16)), dict(zeros=z(3, 6, 2))):
        with pytest.raises(TypeError):
            B.make_q4(**{**dict(codes=codes, scales=scales), **bad})
    for bad in (dict(scales=z(3, 6, 3)), dict(scales=z(2, 6, 2)), dict(scales=z(3, 6, 0)), dict(scales=z(6)),
                dict(zeros=z(3, 6, 1, dtype=u8)), dict(codes=z(3, 32, 6, dtype=u8).transpose(1, 2)),
                dict(codes=z(3, 5, 32, dtype=u8), scales=z(3, 5, 2), act="swiglu")):
        with pytest.raises(ValueError):
            B.make_q4(**{**dict(codes=codes, scales=scales), **bad})
    with pytest.raises(KeyError):
        B.make_q4(codes, scales, code="int8")
