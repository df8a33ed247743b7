"""The checks of the calls around rows sorted by expert under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_host_sanitizers_block.py runs those of the calls
around the experts."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sorted_calls_under_asan_and_ubsan():
    from mxfp4_routed_expert_renorm_amd import build as B
    env = dict(os.environ)
    env.update({
        "MOE_TEST_LIBRARY": B.build_host_sanitized(),
        "LD_PRELOAD": B.asan_runtime(),
        "ASAN_OPTIONS": "detect_leaks=0:detect_odr_violation=0:halt_on_error=1:abort_on_error=0",
        "UBSAN_OPTIONS": "print_stacktrace=1:halt_on_error=1",
    })
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-p", "no:xdist",
           "tests/test_abi_sorted.py", "--deselect",
           "tests/test_abi_sorted.py::test_binding_refuses_tensors_off_the_gpu_and_bad_descriptors"]
    p = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = p.stdout + p.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert p.returncode == 0 and " passed" in out, out[-4000:]
