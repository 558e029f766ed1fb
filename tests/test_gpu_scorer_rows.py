"""Embedding rows and log probabilities on the GPU, with their gradients, against the float64 oracle
(oracle/scorer.py).

Tokens and copied rows are equal.  Numbers stay within bounds derived from float32 arithmetic, u = 2^-24 (half a step,
relative); a rounding to a type is off by eps / 2 relative, or half its smallest subnormal.
  lookup    one product (u), one rounding.
  d_table   n parts, added in any order: at most n u of the sum of their sizes; the scale (u), one rounding.
  softmax   x = (l - m) c: the difference, c (two roundings) and the product, 4 u |x| together; 2^x 1 ulp (2 u); a term of
            Z moves to a new m at most `pieces` times (those of a thread) and 8 times when sums join, 3 u each beside its
            share of 4 u |x|; it is added in a chain of at most 8 pieces + 16.  So Z and S are off, relative to their
            terms, by  r = u (4 away + 3 (pieces + 10) + 8 pieces + 16)  with away the row's largest |x| that matters
            (above 90 the term is below 2^-126).
  logp      2 u |l - m| scale + 3 u |log Z| + r + u |logp|.   H: r (1 + 2 sum p |x|) + 4 u (|log Z| + sum p |x|).
  gradient  p: (4 away + 2 |log Z| + 4) u + r; the bracket d + dH (logp + H): its terms 6 u each, and H's error."""
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
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    with np.errstate(invalid="ignore"):
        err = np.where(got == want, 0.0, np.abs(got - want))   # infinities are equal
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off; worst {np.nanmax(err[bad])} at " \
                          f"{np.argwhere(bad)[0]}, allowed {np.broadcast_to(tol, err.shape)[bad][0]}"


# ---- embedding ---------------------------------------------------------------------------------------

LOOKUPS = [(1, 1, 1), (1, 5, 4096), (3, 7, 250), (64, 100, 128), (65, 1000, 33), (300, 50, 1024), (5, 9, 20000),
           (2500, 3, 8), (2049, 40, 640)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T, V, D", LOOKUPS)
def test_embedding(svt, T, V, D, kind):
    say("embedding", T, V, D, kind)
    rng = np.random.default_rng(T + V + D)
    ids = rng.integers(-2, V + 2, T)
    if T > 4:
        ids[:4] = (-2 ** 62, 2 ** 62, 2 ** 32, V - 1)      # far outside, and one that 32 bits would bring inside
    for shift, scale in ((0, 1.0), (1, -2.7)):
        table = dev(rng.normal(size=(V, D)), ty(kind), shift)
        got = host(svt.svt_embedding(table, dev(ids), scale=scale))
        want = S.embedding(host(table), ids, float(np.float32(scale)))
        exact = scale == 1.0
        near(got, want, 0.0 if exact else (HALF[kind] + U) * np.abs(want) + TINY[kind], "rows")


def grad_ids(rng, T, V, how):
    if how == "spread":
        return rng.integers(-1, V + 1, T)
    if how == "one":
        return np.full(T, V // 2)
    if how == "none":
        return np.full(T, V)
    return np.where(rng.random(T) < 0.6, V - 1, rng.integers(0, max(1, V // 3), T))   # one token for most


GRADS = [(1, 1, 1), (1, 300, 64), (7, 3, 5), (64, 64, 128), (100, 5003, 250), (1000, 37, 24), (1025, 1023, 16),
         (4097, 1025, 40), (8192, 100, 8), (8193, 70000, 12), (9000, 1 << 20, 4), (20000, 600, 32)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("how", ["spread", "one", "most", "none"])
@pytest.mark.parametrize("T, V, D", GRADS)
def test_embedding_backward(svt, T, V, D, how, kind):
    import torch
    say("embedding_backward", T, V, D, how, kind)
    rng = np.random.default_rng(T + V + D)
    ids, scale = grad_ids(rng, T, V, how), 1.7
    d_out = dev(rng.normal(size=(T, D)), ty(kind), T % 3)
    want, size, n = S.embedding_backward(host(d_out), ids, V, float(np.float32(scale)))
    part = U * (n[:, None] + 2) * size
    out = torch.full((V, D), float("nan"), dtype=ty(kind), device="cuda")
    got = svt.svt_embedding_backward(d_out, dev(ids), V, scale=scale, out=out)
    again = svt.svt_embedding_backward(d_out, dev(ids), V, scale=scale)
    near(host(got), want, part + HALF[kind] * (np.abs(want) + part) + TINY[kind] * (n[:, None] > 0), "d_table")
    assert torch.equal(got, again), "the same inputs, other bits"
    old = rng.normal(size=(V, D)).astype(np.float32)
    untouched = np.nan if V > 3 else 0.0
    old[n == 0] = untouched
    total = dev(old, shift=1)
    svt.svt_embedding_backward(d_out, dev(ids), V, scale=scale, out=total, accumulate=True)
    got = host(total)
    assert np.array_equal(got[n == 0], old[n == 0].astype(np.float64), equal_nan=True), "a row that no token names"
    hit = n > 0
    near(got[hit], (want + old)[hit], (part + U * (np.abs(want + old) + part))[hit], "added to float32")


def test_embedding_backward_many_tokens(svt):
    """300,000 tokens, popular and rare, of a table whose keys take two digits: against the float64 sums."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    T, V, D = 300000, 60000, 64
    ids = (torch.rand(T, generator=g, device="cuda", dtype=torch.float64) ** 6 * V).long()
    ids[::97] = V // 2 + 1
    d_out = torch.randn((T, D), generator=g, device="cuda")
    want = torch.zeros((V, D), dtype=torch.float64).index_add_(0, ids.cpu(), d_out.double().cpu())
    size = torch.zeros((V, D), dtype=torch.float64).index_add_(0, ids.cpu(), d_out.double().abs().cpu())
    n = torch.bincount(ids.cpu(), minlength=V).double()[:, None]
    got = host(svt.svt_embedding_backward(d_out, ids, V))
    # chains of at most 256, then one over at most 300000 / 256 chunks
    near(got, want.numpy(), (U * torch.minimum(n, 256 + n / 256 + 2) * size).numpy() + U * want.abs().numpy(), "d_table")


def test_embedding_of_no_tokens(svt):
    import torch
    ids = torch.empty((0,), dtype=torch.int64, device="cuda")
    assert svt.svt_embedding(torch.ones((3, 4), device="cuda"), ids).shape == (0, 4)
    d = svt.svt_embedding_backward(torch.empty((0, 5), device="cuda"), ids, 7, out=torch.ones((7, 5), device="cuda"))
    assert not host(d).any()
    d = svt.svt_embedding_backward(torch.empty((0, 5), device="cuda"), ids, 7, out=torch.ones((7, 5), device="cuda"),
                                   accumulate=True)
    assert host(d).all()


def test_embedding_shapes(svt):
    import torch
    ids = torch.arange(12, device="cuda").view(3, 4) % 5
    table = torch.randn((5, 6), device="cuda")
    out = svt.svt_embedding(table, ids, scale=2.0)
    assert torch.equal(out, 2.0 * table[ids])
    d = svt.svt_embedding_backward(out, ids, 5)
    assert d.shape == (5, 6)


def test_embedding_gradient_by_differences(svt):
    """A sum of squares of the rows: its slope along a direction in the table, against the gradient."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn((50, 8), generator=g, device="cuda")
    way = torch.randn((50, 8), generator=g, device="cuda")
    ids = torch.randint(-1, 51, (200,), generator=g, device="cuda")

    def loss(t):
        return float(svt.svt_embedding(t, ids, scale=0.5).double().square().sum())

    d = svt.svt_embedding_backward(2.0 * svt.svt_embedding(table, ids, scale=0.5), ids, 50, scale=0.5)
    h = 2.0 ** -6
    slope = (loss(table + h * way) - loss(table - h * way)) / (2 * h)
    # the loss is quadratic, so the difference has no error of its own; roundings of t +- h way and of the rows: 8 u of
    # the sum of squares, over h
    assert abs(slope - float((d.double() * way.double()).sum())) <= 8 * U * (loss(table) + loss(way)) * 2 / h


# ---- log probabilities -------------------------------------------------------------------------------

def rows_for(rng, T, V, kind):
    """Logits with the rows that can go wrong."""
    l = 3.0 * rng.normal(size=(T, V))
    shut = rng.random((T, V)) < 0.1
    l[shut] = np.where(rng.random(int(shut.sum())) < 0.5, -np.inf, np.nan)
    low = {"f32": -float(np.finfo(np.float32).max), "f16": -65504.0, "bf16": -3.3895313892515355e38}[kind]
    special = [lambda r: r.fill(-np.inf), lambda r: r.fill(0.25), lambda r: r.fill(low),
               lambda r: r.__setitem__(slice(None), np.sort(rng.normal(size=V))),
               lambda r: r.__setitem__(rng.random(V) < 0.5, low),
               lambda r: r.__setitem__(rng.integers(0, V, 3), np.inf),
               lambda r: r.fill(np.nan),
               lambda r: r.__setitem__(slice(None), np.where(np.arange(V) == V - 1, 0.0, -np.inf)),
               lambda r: r.__setitem__(slice(None), np.repeat(rng.normal(size=V // 7 + 1), 7)[:V])]
    for i, f in enumerate(special[:max(0, T - 1)]):
        f(l[1 + i])
    return l


def in_float32(lp):
    """A log probability below the least float32 (1.6 times a mask of the type's lowest value) rounds to -inf."""
    return np.where(lp < -S.FLT_MAX, -np.inf, lp)


def check_rows(svt, lt, tokens, K, scale, d, dh, kind, name, out=None):
    """Forward and gradient of logits lt against the oracle, row by row."""
    l = host(lt)
    T, V = l.shape
    s32 = float(np.float32(scale))
    got = svt.svt_token_logprobs(lt, dev(tokens), top=K, scale=scale)
    assert len(got) == (5 if K else 3)
    logprobs, entropy = host(got[0]), host(got[1])
    grad = host(svt.svt_token_logprobs_backward(lt, dev(tokens), got[2], got[1], dev(d),
                                                None if dh is None else dev(dh), scale=scale, out=out))
    top_tokens, top_lp = (host(got[3]), host(got[4])) if K else (None, None)
    pieces = -(-V // 512) + 2
    for t in range(T):
        r = S.Row(l[t], s32)
        live = r.away[r.open & (r.away < 90)]
        away = float(live.max()) if live.size else 0.0
        rel = U * (4 * away + 3 * (pieces + 10) + 8 * pieces + 16)

        def lp_tol(lp, a):
            lp, a = np.where(np.isfinite(lp), np.abs(lp), 0.0), np.where(np.isfinite(a), a, 0.0)
            return U * (2 * a + 3 * abs(r.log_z) + lp) + rel

        at = int(tokens[t]) if 0 <= tokens[t] < V else None
        want = 0.0 if at is None else in_float32(r.logp[at])
        near(logprobs[t], want, lp_tol(np.array(want), 0.0 if at is None else r.away[at]), f"{name} row {t} logprob")
        h_tol = rel * (1 + 2 * r.spread) + 4 * U * (abs(r.log_z) + r.spread)
        near(entropy[t], r.entropy, h_tol, f"{name} row {t} entropy")
        if K:
            ids, lp = r.top(K)
            lp = in_float32(lp)
            assert np.array_equal(top_tokens[t], ids), (name, t, top_tokens[t], ids)
            away_of = np.where(ids >= 0, r.away[ids], 0.0)
            near(top_lp[t], lp, lp_tol(lp, away_of), f"{name} row {t} top logprobs")
        hd = 0.0 if dh is None else float(dh[t])
        want = r.backward(at if at is not None else -1, float(d[t]), hd)
        a90 = np.minimum(r.away, 90.0)
        size = abs(float(d[t])) * (at is not None) + abs(hd) * (r.entropy + abs(r.log_z) + a90)
        tol = s32 * r.p * ((U * (4 * a90 + 2 * abs(r.log_z) + 4) + rel + 6 * U) * size + abs(hd) * h_tol)
        tol = tol + HALF[kind] * (np.abs(want) + tol) + TINY[kind] + 2.0 ** -125 * (1 + size)
        if at is not None:
            tol[at] += 2 * U * s32 * abs(float(d[t]))
        near(grad[t], want, tol, f"{name} row {t} gradient")


LOGPROBS = [(1, 1, 1), (1, 2, 2), (11, 7, 7), (10, 8, 3), (12, 9, 0), (13, 63, 16), (10, 64, 1), (11, 511, 16),
            (10, 513, 5), (10, 1000, 0), (10, 1023, 16), (10, 1024, 8), (10, 1025, 16), (12, 2048, 16), (10, 2049, 3),
            (10, 4099, 16), (3, 9001, 2), (1, 4096, 16), (2, 33001, 16), (1, 131072, 8), (10, 20011, 7)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T, V, K", LOGPROBS)
def test_logprobs(svt, T, V, K, kind):
    say("logprobs", T, V, K, kind)
    rng = np.random.default_rng(T * 7 + V + K)
    l = rows_for(rng, T, V, kind)
    lt = dev(l, ty(kind), shift=1)
    tokens = rng.integers(-1, V + 1, T)
    if T > 2:
        tokens[2] = 2 ** 32          # which 32 bits would bring inside
    d, dh = rng.normal(size=T).astype(np.float32), rng.normal(size=T).astype(np.float32)
    check_rows(svt, lt, tokens, K, 1.0, d, dh, kind, "plain")
    if T > 2:
        check_rows(svt, lt, rng.integers(0, V, T), 0, 1.6, d, None, kind, "scaled")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_logprobs_rows_that_go_round(svt, kind):
    """More rows than one grid has, in the form with a wave a row; rows of every part are compared."""
    import torch
    T, V = (1 << 22) + 77, 5
    g = torch.Generator(device="cuda").manual_seed(2)
    lt = torch.randn((T, V), generator=g, device="cuda").to(ty(kind))
    tokens = torch.randint(-1, V, (T,), generator=g, device="cuda")
    lp, h, norms, ids, tlp = svt.svt_token_logprobs(lt, tokens, top=2)
    d = torch.ones(T, device="cuda")
    grad = svt.svt_token_logprobs_backward(lt, tokens, norms, h, d, d)
    pick = [0, 1, 5, 4095, 1 << 20, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, T - 2, T - 1]
    sub = svt.svt_token_logprobs(lt[pick].contiguous(), tokens[pick].contiguous(), top=2)
    for a, b in zip((lp, h, norms, ids, tlp), sub):
        assert torch.equal(a[pick], b)
    check_rows(svt, lt[pick].contiguous(), host(tokens[pick]), 2, 1.0, np.ones(10, np.float32), np.ones(10, np.float32),
               kind, "picked")
    again = svt.svt_token_logprobs_backward(lt[pick].contiguous(), tokens[pick].contiguous(), sub[2], sub[1],
                                            d[:10].contiguous(), d[:10].contiguous())
    assert torch.equal(grad[pick], again)


def test_logprobs_other_alignment_of_the_gradient(svt):
    rng = np.random.default_rng(8)
    for kind in ("f32", "bf16"):
        import torch
        lt = dev(rng.normal(size=(5, 1203)), ty(kind), shift=1)
        out = torch.zeros(5 * 1203 + 2, dtype=ty(kind), device="cuda")[2:].view(5, 1203)
        d = rng.normal(size=5).astype(np.float32)
        check_rows(svt, lt, rng.integers(0, 1203, 5), 3, 0.7, d, d, kind, "shifted", out=out)


def test_logprobs_of_no_rows(svt):
    import torch
    e = torch.empty((0, 9), device="cuda")
    t = torch.empty((0,), dtype=torch.int64, device="cuda")
    lp, h, norms, ids, tlp = svt.svt_token_logprobs(e, t, top=4)
    assert lp.shape == (0,) and norms.shape == (0, 2) and ids.shape == tlp.shape == (0, 4)
    assert svt.svt_token_logprobs_backward(e, t, norms, h, lp).shape == (0, 9)


def test_logprobs_gradient_by_differences(svt):
    """log p and H in float32 along a direction in the logits, by a central difference of the float64 definition, against
    the gradient: the step's own error is its third derivative, at most 8 h^2 here; the gradient is the kernel's."""
    rng = np.random.default_rng(4)
    l, way = rng.normal(size=(6, 40)).astype(np.float32), rng.normal(size=(6, 40))
    tokens = rng.integers(0, 40, 6)
    d, dh = rng.normal(size=6).astype(np.float32), rng.normal(size=6).astype(np.float32)
    lt = dev(l)
    lp, h, norms = svt.svt_token_logprobs(lt, dev(tokens), scale=0.5)
    grad = host(svt.svt_token_logprobs_backward(lt, dev(tokens), norms, h, dev(d), dev(dh), scale=0.5))
    step = 2.0 ** -10
    for t in range(6):
        def f(x):
            r = S.Row(x, 0.5)
            return d[t] * r.logp[tokens[t]] + dh[t] * r.entropy
        slope = (f(l[t] + step * way[t]) - f(l[t] - step * way[t])) / (2 * step)
        size = (abs(d[t]) + 10 * abs(dh[t])) * np.abs(way[t]).max() ** 3
        assert abs(slope - float(grad[t] @ way[t])) <= 8 * step ** 2 * size + 1e-5 * size
