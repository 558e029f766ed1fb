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


# signalling NaNs: the quiet bit is not set
SIGNAL = {"f32": (np.int32, 0x7F800001), "f16": (np.int16, 0x7C01), "bf16": (np.int16, 0x7F81)}


@pytest.mark.parametrize("kind", list(SIGNAL))
@pytest.mark.parametrize("V", [5, 64, 1000, 2048, 131072])
def test_signalling_nans_shut_a_token(svt, V, kind):   # noqa: F811
    """As -inf does, wherever they lie."""
    import torch
    say("signalling", V, kind)
    rng = np.random.default_rng(V)
    T = 3
    l = dev(rng.normal(size=(T, V)), ty(kind))
    bad = rng.random((T, V)) < 0.3
    bad[:, 0], bad[:, V - 1], bad[:, 1] = True, True, False
    bad[2] = True   # a row without an open token
    open_ = l.clone()
    open_[torch.from_numpy(bad).cuda()] = -float("inf")
    bits, value = SIGNAL[kind]
    l.view(torch.int32 if bits is np.int32 else torch.int16)[torch.from_numpy(bad).cuda()] = value
    tokens, d = dev(np.array([1, 0, 1])), dev(np.ones(T, np.float32))
    top = min(4, V)
    a, b = (svt.svt_token_logprobs(t, tokens, top=top, scale=1.5) for t in (l, open_))
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    p, q = (svt.svt_token_logprobs_backward(t, tokens, f[2], f[1], d, d, scale=1.5) for t, f in ((l, a), (open_, b)))
    assert torch.equal(p, q)
