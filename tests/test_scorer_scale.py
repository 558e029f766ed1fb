"""Log probabilities on the host: scales whose product with log2 e would overflow are refused."""
import numpy as np
import pytest

from int8_ivf_ann_amd import svt
from test_scorer_abi import L, P, refused   # noqa: F401 (L is a fixture)

ABOVE = [float(np.nextafter(np.float32(2.0 ** 127), np.float32(np.inf))), 2.4e38, 3e38, float(np.finfo(np.float32).max)]


@pytest.mark.parametrize("scale", ABOVE)
def test_scales_above_the_limit_are_refused(L, scale):   # noqa: F811
    refused(L.svt_token_logprobs(4, 64, 0, svt.SVT_F32, P[0], P[1], scale, P[2], P[3], P[4], None, None, None, 0, None), text="scale")
    refused(L.svt_token_logprobs_backward(4, 64, svt.SVT_F32, P[0], P[1], scale, P[2], P[3], P[4], None, P[6], None), text="scale")
