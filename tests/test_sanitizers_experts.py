"""The host halves of the experts' and the adapters' sources (argument checks,
planning, workspace sizes and launches) under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU.

The sources are compiled for the host alone and linked with stand-ins for the
HIP runtime (tests/sanitize/hip_stub.cpp).  The boundary suites run against
that library, then a sweep of shapes up to the limits: every size is computed
without an overflow, and every accepted call launches grids that a launch can
hold.  Pointers are never dereferenced, and nothing here touches a GPU."""
import os
import re
import subprocess
import sys

from test_sanitizers import CSRC, HIPCC, ROOT, SAN_ENV, _clang_asan_runtime, needs_host_san

SOURCES = ["q4_api.cpp", "q4_experts_api.cpp", "q4_lora_api.cpp", "q4_ragged.hip", "q4_route.hip", "q4_lora.hip"]
STUBS = ["q4_launch_stub.cpp", "hip_stub.cpp"]

_DRIVER = r"""
import ctypes, random, sys
sys.path[:0] = [{root!r}, {tests!r}]
import bit_weight_gemv_amd as q4
q4.LIB_PATH = {lib!r}
import pytest
rc = pytest.main(["-q", "-x", "-s", "-p", "no:cacheprovider", {boundary!r}, {limits!r}])
if rc != 0:
    sys.exit(rc)
from bit_weight_gemv_amd import _base, experts, lora
P = lambda i: (i + 1) << 56          # far apart: the largest operands have 2^48 bytes
L = q4.lib()


def call(m, name, *a):
    s = _base.function(name, m._ARGS)(*a)
    assert L.hipstub_bad() == 0, (name, a)   # a grid that no launch can hold
    return s


rng = random.Random(7)
log = lambda lo, hi: max(lo, min(hi, int(lo * (hi / lo) ** rng.random() + rng.choice((0, 0, 0, 1)))))
ends = lambda lo, hi: rng.choice((lo, hi)) if rng.random() < 0.2 else log(lo, hi)
taken = [0] * 5
for i in range(20000):
    E, M, K = ends(1, 1024), ends(1, 1 << 24), 64 * ends(1, 2048)
    T, R, up = ends(1, 1 << 22), ends(1, 1 << 22), rng.random() < 0.5
    need = call(experts, "q4_gemm_grouped_ws_bytes", E, M, K, T, R, int(up))
    s = call(experts, "q4_gemm_grouped", P(0), P(1), P(2) if up else None, P(3) if up else None, E, M, K, P(4), T, P(5),
             P(6), R, rng.randint(0, 1), P(7), P(8), need, None)
    assert s in (0, 2), s
    taken[0] += s == 0
    r, ad, N = 8 * ends(1, 16), ends(1, 1024) * rng.choice((0, 1, 1, 1)), ends(1, 1 << 22)
    need = call(lora, "q4_gemm_lora_ws_bytes", M, K, N, r, ad)
    s = call(lora, "q4_gemm_lora", P(0), P(1), M, K, P(2), N, P(3), P(4), P(5), P(6), r, ad, 0, P(7), P(8), need, None)
    assert s in (0, 2), s
    taken[1] += s == 0
    need = call(lora, "q4_gemm_lora_backward_ws_bytes", M, K, N, r, ad)
    d = rng.choice(((P(8), P(9), P(10)), (P(8), None, None), (None, P(9), P(10))))
    s = call(lora, "q4_gemm_lora_backward", P(0), P(1), P(2), M, K, P(3), N, P(4), P(5), P(6), P(7), r, ad, *d, P(11), need,
             None)
    assert s in (0, 2), s
    taken[2] += s == 0
    k = ends(1, 16)
    need = call(experts, "q4_route_topk_ws_bytes", T, E, k)
    s = call(experts, "q4_route_topk", P(0), 0, T, E, k, 0, P(1), P(2), P(3), P(4), P(5), P(6), need, None)
    assert s in (0, 2), s
    taken[3] += s == 0
    s = call(experts, "q4_moe_combine", P(0), 1, R, M, P(1), P(2), T, k, 1, P(3), None)
    assert s in (0, 2), s
    taken[4] += s == 0
assert min(taken) > 1000, taken
assert L.hipstub_launches() > 20000, L.hipstub_launches()
print("sweep done")
"""


@needs_host_san
def test_experts_and_adapters_host_code_under_asan_ubsan(tmp_path):
    flags = ["--offload-arch=gfx950", "--offload-host-only", "-std=c++17", "-fPIC", "-g", "-O1",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    objs = []
    for src in [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "tests", "sanitize", s) for s in STUBS]:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run([HIPCC, "-x", "hip", *flags, "-c", src, "-o", objs[-1]], check=True, capture_output=True)
    # The device code that the registration would name is not there.
    names = subprocess.run(["nm", *objs], check=True, capture_output=True, text=True).stdout
    absent = sorted(set(re.findall(r" U (__hip_fatbin\w+)", names)))
    lib = str(tmp_path / "libq4_host_san.so")
    subprocess.run([HIPCC, "-shared", "-no-hip-rt", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
                    "-fsanitize=undefined", "-shared-libsan", *[f"-Wl,--defsym={n}=0" for n in absent], *objs, "-o", lib],
                   check=True, capture_output=True)
    tests = os.path.join(ROOT, "tests")
    driver = tmp_path / "driver.py"
    driver.write_text(_DRIVER.format(root=ROOT, tests=tests, lib=lib,
                                     boundary=os.path.join(tests, "test_boundary_experts_lora.py"),
                                     limits=os.path.join(tests, "test_boundary_experts_lora_limits.py")))
    env = dict(os.environ, LD_PRELOAD=_clang_asan_runtime(), **SAN_ENV)
    r = subprocess.run([sys.executable, str(driver)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "Sanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert "sweep done" in out, out[-2000:]
