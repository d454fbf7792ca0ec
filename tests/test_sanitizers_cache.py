"""The host halves of the cache's sources (argument checks,
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

SOURCES = ["q4_api.cpp", "q4_cache_api.cpp", "q4_cache.hip", "q4_attend.hip"]
STUBS = ["q4_launch_stub.cpp", "hip_stub.cpp"]

_DRIVER = r"""
import ctypes, random, sys
sys.path[:0] = [{root!r}, {tests!r}]
import bit_weight_gemv_amd as q4
q4.LIB_PATH = {lib!r}
import pytest
rc = pytest.main(["-q", "-x", "-s", "-p", "no:cacheprovider", {boundary!r}])
if rc != 0:
    sys.exit(rc)
from bit_weight_gemv_amd import _base, cache
P = lambda i: (i + 1) << 56          # far apart: the largest operands have 2^48 bytes
L = q4.lib()


def call(name, *a):
    s = _base.function(name, cache._ARGS)(*a)
    assert L.hipstub_bad() == 0, (name, a)   # a grid that no launch can hold
    return s


rng = random.Random(7)
log = lambda lo, hi: max(lo, min(hi, int(lo * (hi / lo) ** rng.random() + rng.choice((0, 0, 0, 1)))))
ends = lambda lo, hi: rng.choice((lo, hi)) if rng.random() < 0.2 else log(lo, hi)
taken = [0] * 3
for i in range(20000):
    heads, D, page = ends(1, 1024), 64 * rng.randint(1, 4), 16 << rng.randint(0, 8)
    c = cache.CacheStruct(*[P(20 + x) for x in range(6)], ends(1, (2 ** 31 - 1) // page) if rng.random() < 0.9 else 0, heads, page, D)
    at = ctypes.addressof(c)
    T, qh = ends(1, 1 << 22), heads * ends(1, max(1, 1024 // heads))
    w = heads * D + 8 * ends(1, 1 << 20)
    s = call("q4_cache_append", at, P(0), P(1), rng.randint(0, 1), T, w, w, P(2), P(3), P(4), 16 * rng.randint(0, D // 16), 0, 1.0,
             P(5), qh, qh * D, P(6), None)
    assert s == 0, s
    taken[0] += 1
    s = call("q4_cache_read", at, P(0), T, rng.randint(0, 1), P(1), P(2) if rng.random() < 0.7 else None, None)
    assert s == 0, s
    taken[1] += 1
    B = ends(1, 1 << 22)
    one = rng.random() < 0.3
    if one:
        T = B
    mq = 1 if one else ends(1, 1 << 22)
    need = call("q4_cache_attend_ws_bytes", T, qh, heads, D, B, mq)
    win = rng.choice((0, ends(1, 2 ** 31 - 1)))
    s = call("q4_cache_attend", P(0), T, qh, qh * D, at, P(1), B, ends(1, 1 << 30) // page, P(2), None if one else P(3), mq, 1, win, 0.1,
             rng.randint(0, 1), P(4), P(5), P(9), need, None)
    assert s in (0, 2), s
    assert s == 0 or T * qh > 1 << 29 or B * heads > 1 << 22, (T, qh, heads, D, B, mq)
    taken[2] += s == 0
assert min(taken) > 1000, taken
assert L.hipstub_launches() > 40000, L.hipstub_launches()
print("sweep done")
"""


@needs_host_san
def test_cache_host_code_under_asan_ubsan(tmp_path):
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
                                     boundary=os.path.join(tests, "test_boundary_cache.py")))
    env = dict(os.environ, LD_PRELOAD=_clang_asan_runtime(), **SAN_ENV)
    r = subprocess.run([sys.executable, str(driver)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "Sanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert "sweep done" in out, out[-2000:]
