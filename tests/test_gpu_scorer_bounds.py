"""The trained scorer's operators on the GPU within bounds close enough to see a lost part.  u = 2^-24."""
import numpy as np
import pytest

from gpu_common import say
from oracle import scorer as S
from test_gpu_scorer_gated import HALF, TINY, U, dev, host, near, svt, ty   # noqa: F401 (svt is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [2, 64, 2048, 40000])
def test_logprobs_at_the_largest_scale(svt, V):   # noqa: F811
    """Any difference of these logits is 0 or far, so that p is 1 / n at the n largest and 0 elsewhere; 2 and 1 of them."""
    say("largest scale", V)
    l = np.zeros((2, V), np.float32)
    l[0, [0, V - 1]] = 1.0
    l[1, 1] = 2.0 ** -100
    tokens, scale, one = np.array([V - 1, 1]), 2.0 ** 127, np.ones(2, np.float32)
    lp, H, norms, ids, tlp = svt.svt_token_logprobs(dev(l), dev(tokens), top=2, scale=scale)
    near(host(lp), np.array([-np.log(2), 0.0]), 4 * U, "logp")
    near(host(H), np.array([np.log(2), 0.0]), 4 * U, "entropy")
    assert host(ids).tolist() == [[0, V - 1], [1, 0]]
    near(host(tlp)[:, 0], np.array([-np.log(2), 0.0]), 4 * U, "best")
    d = host(svt.svt_token_logprobs_backward(dev(l), dev(tokens), norms, H, dev(one), scale=scale))
    want = np.zeros((2, V))
    want[0, [0, V - 1]] = -scale / 2, scale / 2
    near(d, want, 16 * U * scale * (np.arange(2)[:, None] == 0) + 16 * U * scale * (np.abs(l) > 0), "d_logits")
