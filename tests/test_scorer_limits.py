"""Gated products of many experts and long sides, embedding gradients of wide rows, on the host: sizes inside the documented ranges are taken, in grids whose
threads along each side stay below 2^32.  The stand-in for the runtime's launch calls (a process of its own) keeps the
largest grid."""
import os
import subprocess
import sys

import pytest

from test_experts_launch import ROOT

STAND_IN = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
int launches; unsigned long long threads_x, blocks; unsigned most_y;
int hipLaunchKernel(const void *f, dim3 g, dim3 b, void **a, size_t lds, void *s) {
  unsigned long long x = (unsigned long long)g.x * b.x, n = (unsigned long long)g.x * g.y * g.z;
  ++launches;
  if (x > threads_x) threads_x = x;
  if (n > blocks) blocks = n;
  if (g.y > most_y) most_y = g.y;
  return 0;
}
int hipGetLastError(void) { return 0; }
int hipPeekAtLastError(void) { return 0; }
"""

CHILD = r"""
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from int8_ivf_ann_amd import svt
L = svt.lib()
threads, blocks = [ctypes.c_ulonglong.in_dll(fake, n) for n in ("threads_x", "blocks")]
R, K, N, M, kind = eval(sys.argv[3])
P = [(i + 1) << 42 for i in range(12)]   # far apart, never read
off = P[11] if M else None
for need in ((1, 1), (1, 0), (0, 1)):
    size = L.svt_gated_linear_backward_workspace_size(R, K, N, M or 1, kind, int(M > 0), 1)
    assert size > 0 and not svt.svt_last_error(), svt.svt_last_error()
    rc = L.svt_gated_linear_backward(R, K, N, M or 1, kind, *P[:6], off, 2, P[6] if need[0] else None,
                                     *(P[7:9] if need[1] else (None, None)), P[9], size, None)
    assert rc == 0, svt.svt_last_error()
size = L.svt_gated_linear_workspace_size(R, K, N, M or 1, kind, int(M > 0), 1)
assert not svt.svt_last_error()
rc = L.svt_gated_linear(R, K, N, M or 1, kind, *P[:3], off, 2, P[6], P[7], P[8], P[9] if size else None, size, None)
assert rc == 0, svt.svt_last_error()
assert 0 < threads.value < 1 << 32, threads.value
print("ok", blocks.value)
"""

# (rows, inputs, outputs, experts, type): of each array there is less than the memory holds
SIZES = [(1000, 64, 131072, 512, 2), (64, 16, 1 << 20, 64, 2), (64, 1, 1 << 20, 512, 2), (64, 1, 1 << 20, 512, 0),
         (1, 1 << 20, 1, 512, 1), (5000, 1, 1 << 20, 512, 2), (2 ** 31 - 1, 1, 1, 0, 1), (2 ** 31 - 1, 1, 1, 512, 1),
         (2 ** 31 - 1, 3, 5, 4, 2), (1 << 20, 1 << 15, 1 << 15, 0, 2), (1 << 14, 4096, 8192, 512, 1)]


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    from int8_ivf_ann_amd import svt
    if not os.path.exists(svt.LIB_PATH):
        from int8_ivf_ann_amd import build
        build.build()
    d = tmp_path_factory.mktemp("limits")
    src, lib, child = d / "stand_in.c", d / "libstand_in.so", d / "child.py"
    src.write_text(STAND_IN)
    child.write_text(CHILD)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    return str(lib), str(child)


@pytest.mark.parametrize("size", SIZES)
def test_sizes_that_fit_the_memory_are_taken(stand_in, size):
    lib, child = stand_in
    r = subprocess.run([sys.executable, child, lib, ROOT, repr(size)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr


def test_sizes_far_beyond_are_refused_by_the_size_call_too():
    from int8_ivf_ann_amd import svt
    L = svt.lib()
    n = 2 ** 31 - 1
    assert L.svt_gated_linear_workspace_size(n, 8, 1 << 20, 1, svt.SVT_F16, 0, 1) == 0
    assert "too many rows" in svt.svt_last_error()
    assert L.svt_gated_linear_backward_workspace_size(n, 1 << 20, 1 << 20, 512, svt.SVT_F16, 1, 1) == 0
    assert "too large" in svt.svt_last_error()


ROWS = r"""
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from int8_ivf_ann_amd import svt
L = svt.lib()
threads, blocks = [ctypes.c_ulonglong.in_dll(fake, n) for n in ("threads_x", "blocks")]
n, V, D, kind = eval(sys.argv[3])
P = [(i + 1) << 42 for i in range(4)]
size = L.svt_embedding_backward_workspace_size(n, V, D)
assert size > 0
for add in (0, 1):
    for shift in (0, 4):   # rows at 16 bytes where the width has it, and at 4
        assert L.svt_embedding_backward(n, V, D, kind, P[0] + shift, P[1], 1.0, add, kind, P[2], P[3], size, None) == 0, svt.svt_last_error()
assert 0 < threads.value < 1 << 32, threads.value
print("ok", blocks.value)
"""


@pytest.mark.parametrize("size", [(4096, 2, 2 ** 24 - 1, 1), (4096, 2, 2 ** 24 - 1, 0), (1, 1, 1, 0), (2 ** 30, 2 ** 31 - 2, 2, 1),
                                  (2 ** 30, 1, 33, 1), (2048, 2048, 2 ** 24, 0)])
def test_embedding_gradients_that_fit_the_memory_are_taken(stand_in, tmp_path, size):
    child = tmp_path / "rows.py"
    child.write_text(ROWS)
    r = subprocess.run([sys.executable, str(child), stand_in[0], ROOT, repr(size)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
