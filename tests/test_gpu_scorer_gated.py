"""Products with a gate on the GPU, and their gradients, against the float64 oracle (oracle/scorer.py).

Bounds from float32 arithmetic, u = 2^-24 (half a step, relative):
  sums       n products of two-byte values are exact in float32, of float32 ones off by u; the additions' roundings, of
             independent sign, grow like their root: (4 sqrt(n + 16) + 4) u of the sum of the parts' sizes (Higham and
             Mary's probabilistic bound with lambda = 4), n the length of the sum.
  activation its slope is below 1.13, so an error of g passes with at most that; its own evaluation is off by
             (g^2 + 2 |g| + 20) u relative (the exponent or the error function's argument is rounded, a few ulp for the
             function); the slope's by 1.3 times as much, absolutely (its two parts are below 1 and 0.3).
  dg, du     rounded to the type before the products: HALF of each, whose effect is summed by size.
Then one rounding of the result."""
import numpy as np
import pytest

from gpu_common import say
from oracle import scorer as S

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}


@pytest.fixture(scope="module")
def svt():
    import torch
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    from int8_ivf_ann_amd import svt as m
    m.lib()
    return m


def ty(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def dev(a, dtype=None, shift=0):
    """The array on the GPU; shift: its storage starts that many elements past an allocation's start."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    if dtype is not None:
        t = t.to(dtype)
    if not shift:
        return t.cuda()
    buf = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
    out = buf[shift:].view(t.shape)
    out.copy_(t)
    return out


def host(t):
    import torch
    torch.cuda.synchronize()
    return t.detach().cpu().to(torch.float64).numpy() if t.is_floating_point() else t.cpu().numpy()


def near(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off; worst {np.nanmax(err[bad])} at " \
                          f"{np.argwhere(bad)[0]}, allowed {np.broadcast_to(tol, err.shape)[bad][0]}"


def sum_tol(n, size):
    return (4 * np.sqrt(n + 16) + 4) * U * size


def act_tol(g):
    return (g * g + 2 * np.abs(g) + 20) * U


def offsets_for(rng, R, M, how):
    if how == "uneven":      # some empty, some long, rows before the first and behind the last
        cut = np.sort(rng.integers(0, R + 1, M + 1))
        if M > 3:
            cut[2] = cut[1]
        return cut.astype(np.int32)
    if how == "one":         # every row on one expert
        o = np.zeros(M + 1, np.int32)
        o[M // 2 + 1:] = R
        return o
    return np.linspace(0, R, M + 1).astype(np.int32)


def check(svt, R, K, N, M, act, kind, shift, how, backward=True, scale=1.0):
    import torch
    rng = np.random.default_rng(R * 31 + K * 7 + N + (M or 0))
    x = dev(scale * rng.normal(size=(R, K)), ty(kind), shift)
    shape = (N, K) if M is None else (M, N, K)
    wg = dev(rng.normal(size=shape) / np.sqrt(K), ty(kind), shift)
    wu = dev(rng.normal(size=shape) / np.sqrt(K), ty(kind), shift)
    o = None if M is None else offsets_for(rng, R, M, how)
    od = None if o is None else dev(o)
    named = np.ones(R, bool) if o is None else (np.arange(R) >= o[0]) & (np.arange(R) < o[-1])
    X, WG, WU = host(x), host(wg).reshape(-1, N, K), host(wu).reshape(-1, N, K)
    h, g, u, sg, su = S.gated(X, WG, WU, act, o)
    outs = [torch.full((R * N + shift,), 7.0, dtype=ty(kind), device="cuda")[shift:].view(R, N) for _ in range(3)]
    got = svt.svt_gated_linear(x, wg, wu, offsets=od, activation=act, keep=True, out=outs[0], out_gate=outs[1],
                               out_up=outs[2])
    alone = svt.svt_gated_linear(x, wg, wu, offsets=od, activation=act)
    keep = [host(t) for t in got]
    assert torch.equal(got[0][torch.from_numpy(named).cuda()], alone[torch.from_numpy(named).cuda()])
    for t in keep:
        assert (t[~named] == 7.0).all(), "rows that no pair names"
    n = named
    tg, tu = sum_tol(K, sg[n]), sum_tol(K, su[n])
    near(keep[1][n], g[n], tg + HALF[kind] * (np.abs(g[n]) + tg) + TINY[kind], "gate")
    near(keep[2][n], u[n], tu + HALF[kind] * (np.abs(u[n]) + tu) + TINY[kind], "up")
    value = S.activation(g[n], act)[0]
    th = (np.abs(u[n]) + tu) * (1.13 * tg + act_tol(g[n]) * np.abs(value)) + np.abs(value) * tu + U * np.abs(h[n])
    near(keep[0][n], h[n], th + HALF[kind] * (np.abs(h[n]) + th) + TINY[kind], "h")
    if not backward:
        return
    dh = dev(rng.normal(size=(R, N)), ty(kind), shift)
    DH, G, UP = host(dh), keep[1], keep[2]
    dx_out = torch.full((R, K), 7.0, dtype=ty(kind), device="cuda")
    dx, dwg, dwu = svt.svt_gated_linear_backward(dh, x, wg, wu, got[1], got[2], offsets=od, activation=act, out_x=dx_out)
    again = svt.svt_gated_linear_backward(dh, x, wg, wu, got[1], got[2], offsets=od, activation=act, need_x=False)
    assert again[0] is None and torch.equal(again[1], dwg) and torch.equal(again[2], dwu)
    only = svt.svt_gated_linear_backward(dh, x, wg, wu, got[1], got[2], offsets=od, activation=act, need_weights=False)
    assert only[1] is None and torch.equal(only[0][torch.from_numpy(n).cuda()], dx[torch.from_numpy(n).cuda()])
    want = S.gated_backward(DH, X, WG, WU, G, UP, act, o)
    value, slope = S.activation(G, act)
    dg, du = DH * UP * slope, DH * value
    eg = np.abs(DH * UP) * 1.3 * act_tol(G) + 3 * U * np.abs(dg)
    eu = np.abs(du) * (act_tol(G) + 2 * U)
    eg = eg + HALF[kind] * (np.abs(dg) + eg) + TINY[kind]
    eu = eu + HALF[kind] * (np.abs(du) + eu) + TINY[kind]
    tx = np.zeros((R, K))
    tw = [np.zeros((len(WG), N, K)) for _ in range(2)]
    for e, a, b in S._rows_of(R, o, len(WG)):
        tx[a:b] = eg[a:b] @ np.abs(WG[e]) + eu[a:b] @ np.abs(WU[e])
        tw[0][e], tw[1][e] = eg[a:b].T @ np.abs(X[a:b]), eu[a:b].T @ np.abs(X[a:b])
        tx[a:b] += sum_tol(2 * N, want[3][a:b] + tx[a:b])
        for q in range(2):
            tw[q][e] += sum_tol(b - a, want[4 + q][e] + tw[q][e])
    got_x = host(dx)
    assert (got_x[~n] == 7.0).all(), "dx of rows that no pair names"
    near(got_x[n], want[0][n], tx[n] + HALF[kind] * (np.abs(want[0][n]) + tx[n]) + TINY[kind], "dx")
    for q, name in enumerate(("dw_gate", "dw_up")):
        near(host((dwg, dwu)[q]).reshape(-1, N, K), want[1 + q], tw[q] + HALF[kind] * (np.abs(want[1 + q]) + tw[q]) + TINY[kind],
             name)


KINDS = ["f32", "f16", "bf16"]
ACTS = ["silu", "gelu", "relu", "none"]

# (rows, inputs, outputs): one row to many, sizes that end inside pieces, steps and tiles
DENSE = [(1, 1, 1), (1, 8, 16), (1, 300, 50), (2, 1000, 24), (16, 64, 64), (17, 33, 17), (33, 130, 100), (64, 256, 130),
         (65, 64, 64), (65, 7, 5), (100, 250, 99), (130, 72, 264), (200, 1, 130), (257, 513, 65), (300, 1032, 40),
         (520, 96, 40)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("i", range(len(DENSE)))
def test_gated_dense(svt, i, kind):
    R, K, N = DENSE[i]
    act = ACTS[i % 4]
    say("gated", R, K, N, act, kind)
    check(svt, R, K, N, None, act, kind, 0, "")
    check(svt, R, K, N, None, ACTS[(i + 1) % 4], kind, 1, "")     # aligned to its elements alone


EXPERTS = [(1, 8, 8, 2, "even"), (7, 40, 24, 5, "uneven"), (64, 128, 64, 32, "uneven"), (64, 96, 40, 3, "one"),
           (300, 72, 136, 4, "uneven"), (513, 64, 72, 7, "even"), (900, 33, 30, 6, "uneven"), (1000, 128, 128, 2, "one"),
           (40, 16, 16, 512, "uneven"), (700, 24, 20, 70, "even")]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("i", range(len(EXPERTS)))
def test_gated_by_expert(svt, i, kind):
    R, K, N, M, how = EXPERTS[i]
    act = ACTS[(i + 2) % 4]
    say("gated by expert", R, K, N, M, how, act, kind)
    check(svt, R, K, N, M, act, kind, i % 2, how)


# tiles enough for the larger cuts: of the forward pass, of dx, of dW
LARGE = [(4100, 72, 1544), (4100, 3100, 40), (70, 2500, 2504), (2050, 200, 900), (1500, 1100, 264)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R, K, N", LARGE)
def test_gated_large(svt, R, K, N, kind):
    say("gated large", R, K, N, kind)
    check(svt, R, K, N, None, "silu", kind, 0, "")


@pytest.mark.parametrize("kind", KINDS)
def test_gated_large_unaligned(svt, kind):
    say("gated large, unaligned", kind)
    check(svt, 4100, 71, 1543, None, "gelu", kind, 1, "")
    check(svt, 70, 2499, 2503, None, "relu", kind, 1, "")
    check(svt, 4100, 1999, 33, 9, "silu", kind, 1, "uneven")


@pytest.mark.parametrize("kind", KINDS)
def test_gated_wide_values(svt, kind):
    """Gates far from 0, where silu and gelu are flat."""
    for act in ("silu", "gelu"):
        check(svt, 40, 64, 48, None, act, kind, 0, "", scale=12.0)
        check(svt, 90, 64, 48, None, act, kind, 0, "", scale=12.0)


def test_gated_of_no_rows(svt):
    import torch
    x, w = torch.empty((0, 24), device="cuda"), torch.ones((2, 8, 24), device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    h, g, u = svt.svt_gated_linear(x, w, w, offsets=o, keep=True)
    assert h.shape == (0, 8)
    dx, dwg, dwu = svt.svt_gated_linear_backward(h, x, w, w, g, u, offsets=o)
    assert dx.shape == (0, 24) and not host(dwg).any() and not host(dwu).any()
    x = torch.ones((5, 24), device="cuda")                # rows, but none for any pair
    h, g, u = svt.svt_gated_linear(x, w, w, offsets=o, keep=True, out=torch.full((5, 8), 3.0, device="cuda"))
    assert (host(h) == 3.0).all()
    dx, dwg, dwu = svt.svt_gated_linear_backward(h, x, w, w, g, u, offsets=o, out_x=torch.full((5, 24), 3.0, device="cuda"))
    assert (host(dx) == 3.0).all() and not host(dwg).any() and not host(dwu).any()


def test_gated_gradient_by_differences(svt):
    """sum(c h) along a direction in x, Wg and Wu: a central difference of the float64 definition, against the gradients."""
    rng = np.random.default_rng(9)
    R, K, N = 30, 20, 12
    x, wg, wu, c = (rng.normal(size=s).astype(np.float32) for s in ((R, K), (N, K), (N, K), (R, N)))
    ways = [rng.normal(size=v.shape) for v in (x, wg, wu)]
    for act in ("silu", "gelu", "none"):
        h, g, u = svt.svt_gated_linear(dev(x), dev(wg), dev(wu), activation=act, keep=True)
        grads = svt.svt_gated_linear_backward(dev(c), dev(x), dev(wg), dev(wu), g, u, activation=act)
        step = 2.0 ** -12

        def f(s):
            a, b, d = x + s * ways[0], wg + s * ways[1], wu + s * ways[2]
            return float(np.sum(c * S.gated(a, b[None], d[None], act)[0]))

        slope = (f(step) - f(-step)) / (2 * step)
        got = sum(float(np.sum(host(a) * b)) for a, b in zip(grads, ways))
        size = sum(float(np.sum(np.abs(host(a) * b))) for a, b in zip(grads, ways))
        # the difference's own error is step^2 / 6 of the third derivative, which stays below 1000 times the slopes' sizes
        assert abs(slope - got) <= (200 * step ** 2 + 1e-5) * size
