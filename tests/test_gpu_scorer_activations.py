"""The gate's activations of float32 rows on the GPU: as close far from 0 as next to it.  u = 2^-24; expf is off by 1 ulp
(2 u relative), erfcf and the reciprocal by 2 u to 4 u, and what their arguments were rounded by is made up for.
  silu   e^-v as a square: 4 u and two roundings, 1 + e^-v and its reciprocal 3 u, the product u: 12 u.  Slope
         s + silu (1 - s): 10 u of s, of 1 - s absolutely, 12 u of silu, the roundings.
  gelu   the integral 7 u, the product u: 10 u.  Slope: 8 u of the integral and 12 u of v times the density."""
import numpy as np
import pytest

from gpu_common import say
from oracle import scorer as S
from test_gpu_scorer_gated import TINY, U, dev, host, near, svt   # noqa: F401 (svt is a fixture)

pytestmark = pytest.mark.gpu

V = np.unique(np.concatenate([np.linspace(-91, 110, 40001), np.linspace(-14, 14, 20001),
                              -np.logspace(-30, 1.9, 2000), np.logspace(-37, 38.5, 2000), -np.logspace(2.1, 38.5, 500)]
                             )).astype(np.float32)


@pytest.mark.parametrize("rows", [1, 40])   # the kernel of few rows, tiles
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_values_and_slopes_far_from_zero(svt, act, rows):   # noqa: F811
    import torch
    say("activation", act, rows)
    v = V.astype(np.float64)
    x = dev(np.ones((rows, 1), np.float32))
    wg, wu = dev(V[:, None]), dev(np.ones((len(V), 1), np.float32))
    h, g, u = svt.svt_gated_linear(x, wg, wu, activation=act, keep=True)
    assert np.array_equal(host(g)[0], v)
    value, slope = S.activation(v, act)
    near(host(h)[rows - 1], value, (12 if act == "silu" else 10) * U * np.abs(value) + TINY["f32"], "value")
    one = torch.zeros_like(h)
    one[0] = 1.0
    _, dwg, dwu = svt.svt_gated_linear_backward(one, x, wg, wu, g, u, activation=act)
    near(host(dwu)[:, 0], value, (12 if act == "silu" else 10) * U * np.abs(value) + TINY["f32"], "value of the gradient")
    if act == "silu":
        s = np.exp(-np.logaddexp(0, -v))
        tol = 10 * U * s + 12 * U * np.abs(value) * (1 - s) + np.abs(value) * (10 * U * s + U) + U * np.abs(slope)
    else:
        tol = 8 * U * np.abs(slope - v * np.exp(-v * v / 2) / np.sqrt(2 * np.pi)) + 12 * U * np.abs(v) * np.exp(-v * v / 2) * 0.4
    near(host(dwg)[:, 0], slope, tol + U * np.abs(slope) + TINY["f32"], "slope")


def test_infinite_gates(svt):   # noqa: F811
    """act(inf) = inf and its slope is 1; a NaN stays one."""
    import torch
    v = torch.tensor([[float("inf")], [float("nan")]], device="cuda")
    x, one = torch.ones((1, 1), device="cuda"), torch.ones((2, 1), device="cuda")
    for act in ("silu", "gelu"):
        h = host(svt.svt_gated_linear(x, v, one, activation=act))[0]
        assert h[0] == np.inf and np.isnan(h[1])
        _, dwg, dwu = svt.svt_gated_linear_backward(torch.ones((1, 2), device="cuda"), x, v, one, v.view(1, 2),
                                                    torch.ones((1, 2), device="cuda"), activation=act)
        assert host(dwu)[0, 0] == np.inf and np.isnan(host(dwu)[1, 0]) and np.isnan(host(dwg)[1, 0])
