"""Launch failures of the routed-expert entry points, on the host: a stand-in for the runtime's launch calls (a few
lines of C, loaded ahead of the HIP runtime in a process of its own) counts the launches and fails the n-th."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_IN = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
int launches, fail_at, pending;
static dim3 grid0, block0; static size_t lds0; static void *stream0;
int hipLaunchKernel(const void *f, dim3 g, dim3 b, void **a, size_t lds, void *s) {
  if (++launches != fail_at) return 0;
  pending = 719;
  return 719;
}
int hipGetLastError(void) { int e = pending; pending = 0; return e; }
int hipPeekAtLastError(void) { return pending; }
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, void *s) { grid0 = g; block0 = b; lds0 = lds; stream0 = s; return 0; }
int __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *lds, void **s) { *g = grid0; *b = block0; *lds = lds0; *s = stream0; return 0; }
"""

CHILD = r"""
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from int8_ivf_ann_amd import svt
L = svt.lib()
count, fail, pending = [ctypes.c_int.in_dll(fake, n) for n in ("launches", "fail_at", "pending")]
P = [0x10000000 + (i << 28) for i in range(8)]
w = [svt.svt_quant_weights(1, 32, 64, 32, svt.SVT_F16, z, 0x70000000 + (8 << 28), 1 << 28) for z in (0, 1)]
CALLS = {
    "route": (1, lambda: L.svt_route(4, 8, 2, 0, P[0], 1, P[1], P[2], None)),
    "route_backward": (1, lambda: L.svt_route_backward(4, 8, 2, 0, P[0], 1, P[1], P[2], P[3], P[4], None)),
    "sort_one": (1, lambda: L.svt_expert_sort(64, 2, 8, P[0], P[1], P[2], P[3], None, 0, None)),
    "sort_two": (2, lambda: L.svt_expert_sort(100000, 2, 8, P[0], P[1], P[2], P[3], P[5], 1 << 20, None)),
    "dispatch": (1, lambda: L.svt_expert_dispatch(4, 2, 24, 1, P[0], P[1], P[2], None)),
    "combine": (1, lambda: L.svt_expert_combine(4, 2, 24, 1, P[0], P[1], P[3], P[2], None)),
    "combine_backward": (1, lambda: L.svt_expert_combine_backward(4, 2, 24, 1, P[0], P[1], P[2], P[3], P[4], P[5], None)),
    "pack": (2, lambda: L.svt_quant_pack(ctypes.byref(w[0]), P[0], P[1], None, None)),
    "pack_zeros": (3, lambda: L.svt_quant_pack(ctypes.byref(w[1]), P[0], P[1], P[2], None)),
    "linear": (1, lambda: L.svt_quant_linear(4, 1, P[0], ctypes.byref(w[0]), P[1], None, 0, 1, P[2], None)),
}
n, call = CALLS[sys.argv[3]]
for at in range(n + 1):
    count.value, fail.value, pending.value = 0, at, 0
    rc = call()
    assert rc == (svt.SVT_EDEVICE if at else svt.SVT_OK), (at, rc, svt.svt_last_error())
    assert count.value == (at if at else n), f"launch {at} of {n} failed, {count.value} were made"
    assert pending.value == 0, "the call reports its own failure and leaves none behind"
    assert bool(svt.svt_last_error()) == bool(at)
# a failure of some other call, not read yet: none of this call's, and still the caller's to read
count.value, fail.value, pending.value = 0, 0, 2
rc = call()
assert rc == svt.SVT_OK and count.value == n, (rc, count.value, svt.svt_last_error())
assert pending.value == 2
print("ok")
"""

CALLS = ["route", "route_backward", "sort_one", "sort_two", "dispatch", "combine", "combine_backward", "pack",
         "pack_zeros", "linear"]


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    from int8_ivf_ann_amd import svt
    if not os.path.exists(svt.LIB_PATH):
        from int8_ivf_ann_amd import build
        build.build()
    d = tmp_path_factory.mktemp("launch")
    src, lib, child = d / "stand_in.c", d / "libstand_in.so", d / "child.py"
    src.write_text(STAND_IN)
    child.write_text(CHILD)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    return str(lib), str(child)


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_ends_the_call(stand_in, name):
    lib, child = stand_in
    r = subprocess.run([sys.executable, child, lib, ROOT, name], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
