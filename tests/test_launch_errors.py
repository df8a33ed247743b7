"""A launch that fails is reported, and no call asks for more threads than a launch can have
(no GPU): the calls around rows sorted by expert in a process whose launches end in a
stand-in, so that none reaches a device.  Arguments pass the checks, addresses are invented."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Launches are counted, fail where the process asks for it or where a dimension has 2^32
# threads or more, 65536 workgroups beyond the first dimension, or none.
STAND_IN = r"""
#include <cstddef>
#include <cstdint>
struct Dim { uint32_t x, y, z; };
struct Call { Dim grid, block; size_t lds; void* stream; };
static int last = 0;
static Call call;
extern "C" {
int stand_in_fails = 1;
long stand_in_launches = 0;
static int launch(Dim g, Dim b) {
  ++stand_in_launches;
  const uint64_t n[3] = {(uint64_t)g.x * b.x, (uint64_t)g.y * b.y, (uint64_t)g.z * b.z};
  bool bad = stand_in_fails || g.y > 65535 || g.z > 65535;
  for (uint64_t v : n) bad = bad || v == 0 || v >> 32;
  return last = bad ? 9 : 0;  // hipErrorInvalidConfiguration
}
int __hipPushCallConfiguration(Dim g, Dim b, size_t lds, void* s) { call = {g, b, lds, s}; return 0; }
int __hipPopCallConfiguration(Dim* g, Dim* b, size_t* lds, void** s) {
  *g = call.grid, *b = call.block, *lds = call.lds, *s = call.stream;
  return 0;
}
int hipLaunchKernel(const void*, Dim g, Dim b, void**, size_t, void*) { return launch(g, b); }
int hipExtLaunchKernel(const void*, Dim g, Dim b, void**, size_t, void*, void*, void*, int) { return launch(g, b); }
int hipGetLastError() { const int e = last; last = 0; return e; }
}
"""

CHILD = r"""
import ctypes, itertools, sys
stand_in = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # before the library: its launches come here
from mxfp4_routed_expert_renorm_amd import binding as B
lib, EHIP = B.load(), 5
launches, fails = ctypes.c_long.in_dll(stand_in, "stand_in_launches"), ctypes.c_int.in_dll(stand_in, "stand_in_fails")
fails.value = int(sys.argv[2])
p = lambda i: ctypes.c_void_p((i + 1) << 45)
def call(name, *args):
    before = launches.value
    st = getattr(lib, name)(*args, None)
    assert launches.value > before, f"{name} {args}: not launched: {st}, {lib.moe_last_error().decode()}"
    if fails.value:
        assert st == EHIP and b"launch failed" in lib.moe_last_error(), f"{name} {args}: status {st}"
    else:
        assert st == 0, f"{name} {args}: {lib.moe_last_error().decode()}"
most = 1 << 20
for T, k, H in ((1, 1, 1), (16, 8, 4096), (6144, 1, 65536), (4096, 8, 64), (most, 1, 65536), (1 << 14, 64, 65536)):
    for t in (B.MOE_F32, B.MOE_BF16):
        n = B.moe_permute_scratch_bytes(T, k, 1024)
        call("moe_permute", p(0), t, T, k, H, 1024, p(1), p(2), p(3), p(4), p(5), p(6), n)
for T, k, H in itertools.product((1, 777, most), (1, 64), (1, 512, 2047, 32256, 32257, 65536)):
    call("moe_unpermute", p(0), 0, 64, p(1), None, None, T, k, H, p(2), 0)
    call("moe_unpermute_grad", p(0), 0, p(1), 0, 64, p(2), None, T, k, H, p(3), p(4))
for E, T, scoring in itertools.product((1, 256, 512, 1024), (1, most), ("sigmoid", "softmax")):
    r = B.make_router(E, 1, scoring=scoring, renorm=False)
    call("moe_route_grad", ctypes.byref(r), p(0), 0, T, p(1), p(2), p(3), p(4), 0)
for (code, st), act, (K, group), N in itertools.product(
        ((B.Q4_INT4, B.MOE_BF16), (B.Q4_FP4, B.SCALE_E8M0), (B.Q4_FP4, B.MOE_F32)), (B.Q4_LINEAR, B.Q4_SWIGLU),
        ((512, 32), (512, 128), (160, 32)), (1, 2048, 65536)):
    q = B.moe_q4(K, N, 1024, group, code, act, st, p(0).value, p(1).value, None, 1 << 27, 1 << 27, 0)
    for T, xt in itertools.product((1, 4096, most), (B.MOE_F32, B.MOE_BF16)):  # both forms
        call("moe_q4_linear", ctypes.byref(q), p(2), xt, T, p(3), 0)
        call("moe_q4_grouped", ctypes.byref(q), p(2), xt, T, p(4), p(3), 0)
print("done", launches.value)
"""


def _child(tmp_path, fails):
    src, so = tmp_path / "stand_in.cpp", tmp_path / "stand_in.so"
    src.write_text(STAND_IN)
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-o", str(so), str(src)], check=True)
    p = subprocess.run([sys.executable, "-c", CHILD, str(so), str(fails)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0 and "done" in p.stdout, (p.stdout + p.stderr)[-3000:]


def test_failed_launches_are_reported(tmp_path):
    _child(tmp_path, 1)


def test_launches_fit_the_device_up_to_the_largest_sizes(tmp_path):
    _child(tmp_path, 0)
