"""The trained scorer's operators on the GPU within bounds close enough to see a lost part.  u = 2^-24."""
import numpy as np
import pytest

from gpu_common import say
from oracle import scorer as S
from test_gpu_scorer_gated import HALF, TINY, U, act_tol, dev, host, near, sum_tol, svt, ty   # noqa: F401 (svt is a fixture)

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


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n, D", [(100000, 24), (65536, 1024), (4097, 130), (33, 7)])
def test_one_token_many_times(svt, n, D, kind):   # noqa: F811
    """Sums of one sign.  Places of a chunk (8 at these sizes, 16 for 65536 x 1024, whose 512 columns fill a wave: n / 4096)
    are added one after the other, then a 16th of the chunks by each wave, then the 16 waves' sums: k additions in a chain,
    (k - 1) u of the sum.  A lost chunk would be at least 8 / n of it, more than the bound.  Whole numbers below 2^24 / n in
    size are added exactly."""
    import torch
    say("one token", n, D, kind)
    per = 16 if D == 1024 else 8
    chain = per + -(-(-(-n // per)) // 16) + 16
    assert chain * U < per / n
    ids = torch.full((n,), 2, device="cuda")
    d = torch.full((n, D), 0.7, device="cuda").to(ty(kind))
    got = host(svt.svt_embedding_backward(d, ids, 5, out_dtype=ty("f32")))
    near(got[2], n * float(d[0, 0]), chain * U * n * float(d[0, 0]), "sum")
    assert not got[[0, 1, 3, 4]].any()
    d = torch.randint(-9, 10, (n, D), device="cuda").to(ty(kind))
    got = svt.svt_embedding_backward(d, ids, 5, out_dtype=ty("f32"))
    assert torch.equal(got[2].double(), d.double().sum(0)) and not host(got)[[0, 1, 3, 4]].any()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_the_longest_row_whole(svt, kind):   # noqa: F811
    """2^30 tokens, equal but for three that hold a millionth of the sum: 512 workgroups of 256 threads add 1024 pieces of 8
    each.  A thread's sum is off by n u / 2 with n = 1024 pieces, one after the other, and 8 u within a piece; joins of lanes,
    waves and splits 30, the exponentials and the logarithm 16: 566 u = 3.4e-5.  A lost split would be 2e-3 of log Z's
    argument."""
    import torch
    say("longest, whole", kind)
    V = 1 << 30
    l = torch.zeros((1, V), dtype=ty(kind), device="cuda")
    places, values = [3, V // 2 + 1, V - 1], np.array([3.0, 2.0, 4.0])
    l[0, places] = torch.tensor(values, dtype=torch.float32, device="cuda").to(ty(kind))
    tokens = torch.tensor([V - 1], device="cuda")
    lp, H, nm, ids, tlp = svt.svt_token_logprobs(l, tokens, top=4)
    z = V - 3 + np.exp(values).sum()
    p, p0 = np.exp(values) / z, 1 / z
    bound = (1024 / 2 + 8 + 30 + 16) * U
    assert host(ids)[0].tolist() == [V - 1, 3, V // 2 + 1, 0]
    # beside Z's relative error: roundings of log Z (20.8) and of the difference
    near(host(lp)[0], np.log(p[2]), bound + 64 * U, "logp")
    near(host(tlp)[0], np.log([p[2], p[0], p[1], p0]), bound + 64 * U, "alternatives")
    # H = log Z + 4 - sum p x': the second part is 4, off by twice the bound relative
    near(host(H)[0], -np.sum(p * np.log(p)) - (V - 3) * p0 * np.log(p0), bound * (1 + 2 * 4) + 64 * U, "entropy")
    d = svt.svt_token_logprobs_backward(l, tokens, nm, H, torch.ones(1, device="cuda"))
    rel = bound + 64 * U + HALF[kind]   # 64: the roundings of x - log2 Z (30) and of 2^x
    for i, w in ((3, -p[0]), (V // 2 + 1, -p[1]), (V - 1, 1 - p[2])):
        near(np.float64(d[0, i].item()), w, rel * abs(w), f"d {i}")
    d[0, places] = d[0, 0].clone()
    assert torch.equal(d.min(), d.max())
    near(np.float64(d[0, 0].item()), -p0, rel * p0, "the others")


def rounded(v, error, kind):
    """v rounded to the type, and how far off that is where v is only known within error: 0 but next to a border."""
    import torch

    def to(a):
        return torch.from_numpy(a).to(torch.float32).to(ty(kind)).double().numpy()

    r = to(v)
    return r, np.maximum(to(v + error) - r, r - to(v - error))


# (rows, inputs, outputs, matrices)
GRADIENTS = [(300, 200, 1000, 0), (64, 2000, 4000, 0), (2000, 64, 72, 0), (1500, 96, 640, 5), (70, 33, 3000, 2)]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "none"])
@pytest.mark.parametrize("R, K, N, M", GRADIENTS)
def test_gradients_round_dg_and_du_once(svt, R, K, N, M, act, kind):   # noqa: F811
    """dx and dW against the definition with dg and du rounded to the type, as documented: what is left are the float32 sums,
    one rounding of the result, and dg or du that lie within their own float32 error of a border between two values."""
    say("rounded once", R, K, N, M, act, kind)
    rng = np.random.default_rng(R + K + N)
    E = max(M, 1)
    shape = (M, N, K) if M else (N, K)
    x, dh, g, u = (dev(rng.normal(size=(R, n)), ty(kind)) for n in (K, N, N, N))
    wg, wu = (dev(rng.normal(size=shape) / np.sqrt(K), ty(kind)) for _ in range(2))
    o = np.linspace(0, R, M + 1).astype(np.int32) if M else None
    dx, dwg, dwu = svt.svt_gated_linear_backward(dh, x, wg, wu, g, u, offsets=None if o is None else dev(o), activation=act)
    X, DH, G, UP = host(x), host(dh), host(g), host(u)
    W = [host(w).reshape(E, N, K) for w in (wg, wu)]
    value, slope = S.activation(G, act)
    parts = (DH * UP * slope, DH * value)
    if act == "none":   # products of two values of the type, exact in float32
        errors = (np.zeros_like(DH), np.zeros_like(DH))
    else:
        errors = (np.abs(DH * UP) * 1.3 * act_tol(G) + 3 * U * np.abs(parts[0]), np.abs(parts[1]) * (act_tol(G) + 2 * U))
    (dg, eg), (du, eu) = (rounded(v, e, kind) for v, e in zip(parts, errors))
    for e in range(E):
        r = slice(o[e], o[e + 1]) if M else slice(0, R)
        size = np.abs(dg[r]) @ np.abs(W[0][e]) + np.abs(du[r]) @ np.abs(W[1][e])
        near_by = eg[r] @ np.abs(W[0][e]) + eu[r] @ np.abs(W[1][e])
        want, tol = dg[r] @ W[0][e] + du[r] @ W[1][e], near_by + sum_tol(2 * N, size)
        near(host(dx)[r], want, tol + HALF[kind] * (np.abs(want) + tol) + TINY[kind], "dx")
        assert np.median(tol / size) < 0.1 * HALF[kind]   # close: dg and du rounded anyhow would be allowed HALF of it
        for got, d, err, name in ((dwg, dg, eg, "dw_gate"), (dwu, du, eu, "dw_up")):
            want = d[r].T @ X[r]
            tol = err[r].T @ np.abs(X[r]) + sum_tol(r.stop - r.start, np.abs(d[r]).T @ np.abs(X[r]))
            near(host(got).reshape(E, N, K)[e], want, tol + HALF[kind] * (np.abs(want) + tol) + TINY[kind], name)
