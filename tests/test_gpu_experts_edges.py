"""Routed-expert operators on the GPU at the ends of their ranges, against the float64 oracle.  u = 2^-24."""
import numpy as np
import pytest

from gpu_common import say
from oracle import experts as X
from test_gpu_experts import HALF, TINY, U, dev, host, near, ty

pytestmark = pytest.mark.gpu
FLT_MAX = np.finfo(np.float32).max


@pytest.fixture(scope="module")
def svt():
    import torch
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    from int8_ivf_ann_amd import svt as m
    m.lib()
    return m


# ---- router ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E, K", [(3, 2), (8, 8), (9, 4), (40, 12), (512, 3)])
def test_route_plus_infinity_ties_with_the_largest_float(svt, E, K, renorm):
    """+inf counts as the largest finite float32: the lower expert of the two comes first, with equal weights."""
    say("ties", E, K, renorm)
    l = np.zeros((4, E), np.float32)
    l[0, [0, E - 1]] = FLT_MAX, np.inf
    l[1, [0, E - 1]] = np.inf, FLT_MAX
    l[2, E // 2:] = np.inf
    l[2, :E // 2] = FLT_MAX
    l[3, [1, E - 1]] = np.nextafter(FLT_MAX, np.float32(0)), np.inf   # a step below is below
    ids, w = svt.svt_route(dev(l), K, renormalise=renorm)
    rid, rw, _ = X.route(l, K, renorm)
    assert np.array_equal(host(ids), rid)
    near(host(w), rw, 32 * U * rw, "weights")   # differences of 0 or past every exponential: 31 u, as everywhere
