"""Refusals of buffers that overlap (no GPU): workgroups of the calls around the
experts write rows while others still read theirs, so an output shares memory with
an input only where it is that input's buffer and the header allows it.

The addresses are invented: every call here has to be refused before a launch.  The
calls in place that are allowed run in the GPU's tests."""
import ctypes

import pytest

from mxfp4_routed_expert_renorm_amd import binding as B
from tests.test_abi_block import EINVAL, _norm, _st, lib  # noqa: F401

BASE = 1 << 20
FAR = [BASE + (i << 20) for i in range(8)]  # a MiB apart


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _shifts(size, other):
    """Starts of a buffer of `size` bytes that overlap one of `other` bytes at 0, but for the same start."""
    return sorted({-(size - 4), -4, 4, other - 4} - {0})


@pytest.mark.parametrize("ot,size", [(0, 512), (1, 256)])
def test_norm_in_overlaps(lib, ot, size):  # noqa: F811
    n = _norm(pre_w=FAR[3], wt=0)
    ref = ctypes.byref(n)
    for d in _shifts(size, 512):
        st, msg = _st(lib, "moe_norm_in", ref, _p(FAR[0]), 0, 2, _p(FAR[0] + d), ot, None)
        assert st == EINVAL and "overlap" in msg, d
    for d in _shifts(size, 256) + [0]:
        st, msg = _st(lib, "moe_norm_in", ref, _p(FAR[0]), 0, 2, _p(FAR[3] + d), ot, None)
        assert st == EINVAL and "overlap" in msg, d


@pytest.mark.parametrize("which", ["out", "next_out"])
def test_norm_out_overlaps(lib, which):  # noqa: F811
    n, nxt = _norm(post_w=FAR[5], gate=3), _norm(pre_w=FAR[6])
    at = {"y": FAR[0], "residual": FAR[1], "gate": FAR[2], "out": FAR[3], "next_out": FAR[4]}
    for other, size in (("y", 512), ("residual", 512), ("gate", 512), (FAR[5], 256), (FAR[6], 256),
                        ("next_out" if which == "out" else "out", 512)):
        start = at[other] if isinstance(other, str) else other
        for d in _shifts(512, size) + ([] if other in ("y", "residual") else [0]):
            a = dict(at)
            a[which] = start + d
            st, msg = _st(lib, "moe_norm_out", ctypes.byref(n), _p(a["y"]), 0, _p(a["residual"]), _p(a["gate"]), 0, 2,
                          _p(a["out"]), 0, ctypes.byref(nxt), _p(a["next_out"]), 0, None)
            assert st == EINVAL and ("overlap" in msg or "buffer" in msg), (other, d, msg)


@pytest.mark.parametrize("which", ["ids", "w"])
def test_route_overlaps(lib, which):  # noqa: F811
    r = B.make_router(64, 4)
    at = {"logits": FAR[0], "bias": FAR[1], "ids": FAR[2], "w": FAR[3]}
    for other, size in (("logits", 2048), ("bias", 256), ("w" if which == "ids" else "ids", 128)):
        for d in _shifts(128, size) + [0]:
            a = dict(at)
            a[which] = at[other] + d
            st, msg = _st(lib, "moe_route_groups", ctypes.byref(r), _p(a["logits"]), 0, _p(a["bias"]), 8, _p(a["ids"]),
                          _p(a["w"]), None)
            assert st == EINVAL and "overlap" in msg, (other, d)


def test_lora_overlaps(lib):  # noqa: F811
    m = B.moe_lora(64, 32, 8, 4, FAR[4], FAR[5], FAR[6], FAR[7])
    at = {"x": (FAR[0], 3 * 64 * 2), "ids": (FAR[1], 12), "base": (FAR[2], 3 * 32 * 2), "a": (FAR[4], 4 * 8 * 64 * 2),
          "b": (FAR[5], 4 * 32 * 8 * 2), "scale": (FAR[6], 16), "ranks": (FAR[7], 16)}
    for other, (start, size) in at.items():
        for d in _shifts(192, size) + ([] if other == "base" else [0]):
            st, msg = _st(lib, "moe_lora_add", ctypes.byref(m), _p(FAR[0]), 1, 3, _p(FAR[1]), _p(FAR[2]), _p(start + d), 1,
                          None)
            assert st == EINVAL and ("overlap" in msg or "may not be x" in msg), (other, d)
