"""The trained scorer's operators on the GPU at the ends of their ranges, captured, on other streams and together, against
the float64 oracle.  u = 2^-24."""
import numpy as np
import pytest

from gpu_common import say
from oracle import experts as X
from oracle import scorer as S
from test_gpu_scorer_gated import HALF, TINY, U, act_tol, check, dev, host, near, sum_tol, ty

pytestmark = pytest.mark.gpu
FLT_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def svt():
    import torch
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    from int8_ivf_ann_amd import svt as m
    m.lib()
    return m


# ---- values ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
def test_activations_over_their_range(svt, act):
    """One product of one input: g = v and u = 1 exactly, so h is the activation, and with dh = 1 the weights' and x's
    gradients are its value and slope."""
    import torch
    say("range", act)
    v = np.unique(np.concatenate([np.linspace(-110, 110, 4001), np.linspace(-3, 3, 2001), -np.logspace(-30, 2, 200), [-87.5, -88, -88.5]]))
    v = v.astype(np.float32)
    x = dev(np.ones((1, 1), np.float32))
    wg, wu = dev(v[:, None]), dev(np.ones((len(v), 1), np.float32))
    h, g, u = svt.svt_gated_linear(x, wg, wu, activation=act, keep=True)
    assert np.array_equal(host(g)[0], v.astype(np.float64))
    value, slope = S.activation(v.astype(np.float64), act)
    near(host(h)[0], value, (act_tol(v) + U) * np.abs(value) + TINY["f32"], "value")
    _, dwg, dwu = svt.svt_gated_linear_backward(torch.ones_like(h), x, wg, wu, g, u, activation=act)
    near(host(dwu)[:, 0], value, (act_tol(v) + 2 * U) * np.abs(value) + TINY["f32"], "du")
    near(host(dwg)[:, 0], slope, 1.3 * act_tol(v) + 3 * U * np.abs(slope) + TINY["f32"], "slope")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R", [1, 40, 700])
def test_rows_of_other_experts_do_not_reach_a_row(svt, R, kind):
    """Rows that no expert names, and whole experts' rows, of NaN and infinities; the workspace too.  What the others get is
    what they get without them."""
    import torch
    say("neighbours", R, kind)
    rng = np.random.default_rng(R)
    K, N, M = 77, 45, 5
    n = R + 2 * R + 30
    o = np.array([7, 7 + R, 7 + 2 * R, 7 + 2 * R, 7 + 3 * R, 7 + 3 * R], np.int32)
    bad = np.zeros(n, bool)
    bad[:7] = bad[7 + R:7 + 2 * R] = bad[7 + 3 * R:] = True

    def make(shape, rows_bad):
        a = rng.normal(size=shape)
        b = a.copy()
        if rows_bad:
            b[bad] = rng.choice([np.nan, np.inf, -np.inf], (int(bad.sum()), shape[1]))
            a[bad] = 0
        return dev(a, ty(kind)), dev(b, ty(kind))

    x, xb = make((n, K), True)
    dh, dhb = make((n, N), True)
    wg, _ = make((M, N, K), False)
    wu, _ = make((M, N, K), False)
    od = dev(o)
    wgb, wub = wg.clone(), wu.clone()
    wgb[2], wub[2], wgb[4], wub[4] = float("nan"), float("inf"), float("inf"), float("nan")   # experts without rows
    good = torch.from_numpy(~bad).cuda()
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    h, g, u = svt.svt_gated_linear(x, wg, wu, offsets=od, keep=True)
    hb, gb, ub = svt.svt_gated_linear(xb, wgb, wub, offsets=od, keep=True, workspace=ws)
    for a, b in ((h, hb), (g, gb), (u, ub)):
        assert torch.isfinite(a[good]).all() and torch.equal(a[good], b[good])
    for t in (gb, ub):
        t[torch.from_numpy(bad).cuda()] = float("nan")
    ws.fill_(255)
    d = svt.svt_gated_linear_backward(dh, x, wg, wu, g, u, offsets=od)
    db = svt.svt_gated_linear_backward(dhb, xb, wgb, wub, gb, ub, offsets=od, workspace=ws)
    assert torch.isfinite(d[0][good]).all() and torch.equal(d[0][good], db[0][good])
    for q in (1, 2):
        for e in (0, 2, 3, 4):
            assert torch.isfinite(d[q][e]).all() and torch.equal(d[q][e], db[q][e]), (q, e)


def test_falling_offsets_stay_in_bounds(svt):
    """Offsets are ascending; ends that fall give no defined results, but nothing outside the outputs' and the workspace's
    own bytes is written."""
    import torch
    say("falling")
    rng = np.random.default_rng(1)
    for R, K, N, M in ((600, 40, 24, 9), (5000, 33, 100, 60), (30, 64, 16, 8)):
        o = dev(np.array([0, R] * ((M + 1) // 2) + [R // 2] * ((M + 1) % 2) + [], np.int32)[:M + 1])
        assert o.numel() == M + 1
        f = lambda *s: dev(rng.normal(size=s), torch.bfloat16)
        x, dh, wg, wu = f(R, K), f(R, N), f(M, N, K), f(M, N, K)
        need = svt.svt_gated_linear_backward_workspace_size(R, K, N, M, svt.SVT_BF16, True, True)
        need += -need % 16
        buf = torch.full((need + (1 << 20),), 77, dtype=torch.uint8, device="cuda")
        outs = [torch.full((n + 4096,), 7.0, dtype=torch.bfloat16, device="cuda") for n in (R * K, M * N * K, M * N * K)]
        v = [outs[0][:R * K].view(R, K), outs[1][:M * N * K].view(M, N, K), outs[2][:M * N * K].view(M, N, K)]
        svt.svt_gated_linear_backward(dh, x, wg, wu, dh, dh, offsets=o, out_x=v[0], out_gate=v[1], out_up=v[2], workspace=buf[:need])
        svt.svt_gated_linear(x, wg, wu, offsets=o)
        assert (buf[need:] == 77).all()
        for t, n in zip(outs, (R * K, M * N * K, M * N * K)):
            assert (t[n:] == 7.0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["uneven", "one", "even"])
@pytest.mark.parametrize("R, K, N, M", [(9000, 40, 24, 70), (20000, 24, 20, 3), (6000, 100, 33, 130)])
def test_long_experts_are_cut(svt, R, K, N, M, how, kind):
    """Few and many experts of thousands of rows, whose weights' gradients are sums of blocks."""
    say("cut", R, K, N, M, how, kind)
    need = svt.svt_gated_linear_backward_workspace_size(R, K, N, M, svt.SVT_F32, True, True)
    assert need > 2 * R * ((4 * N + 15) // 16 * 16)   # there are parts
    check(svt, R, K, N, M, "silu", kind, 0, how)


@pytest.mark.parametrize("kind, least", [("bf16", -133), ("f16", -24), ("f32", -133)])
@pytest.mark.parametrize("R", [1, 40, 300])
def test_gated_subnormal_values(svt, R, kind, least):
    """Inputs below the smallest normal number count in full, against weights that bring them back up."""
    say("subnormal", R, kind)
    rng = np.random.default_rng(R)
    K, N = 70, 40
    low = {"f16": 2.0 ** -14, "bf16": 2.0 ** -126, "f32": 2.0 ** -126}[kind]
    x = dev(rng.integers(-63, 64, (R, K)) * 2.0 ** least, ty(kind))
    assert np.abs(host(x)).max() < low and np.abs(host(x)).max() > 0
    up = 2.0 ** (14 if kind == "f16" else 124)
    wg, wu = (dev(rng.integers(-7, 8, (N, K)) * up / 8, ty(kind)) for _ in range(2))
    h, g, u = (host(t) for t in svt.svt_gated_linear(x, wg, wu, activation="none", keep=True))
    rh, rg, ru, sg, su = S.gated(host(x), host(wg)[None], host(wu)[None], "none")
    near(g, rg, sum_tol(K, sg) + HALF[kind] * np.abs(rg), "gate")
    near(u, ru, sum_tol(K, su) + HALF[kind] * np.abs(ru), "up")


@pytest.mark.parametrize("V", [5, 64, 1000, 40000, 131072])
def test_logprobs_infinities_and_ties(svt, V):
    """+inf counts as the largest finite float32, and ties with it; the lower token comes first."""
    say("ties", V)
    l = np.full((4, V), -5.0, np.float32)
    l[0, [1, V - 1]] = FLT_MAX, np.inf
    l[1, [1, V - 1]] = np.inf, FLT_MAX
    l[2, [0, V - 1]] = np.nextafter(np.float32(FLT_MAX), np.float32(0)), np.inf
    l[3] = -np.inf
    l[3, V // 2] = -FLT_MAX
    K = 4
    lp, H, nm, ids, tlp = svt.svt_token_logprobs(dev(l), dev(np.array([1, V - 1, V - 1, V // 2])), top=K)
    for t in range(4):
        r = S.Row(l[t], 1.0)
        rid, rlp = r.top(K)
        assert np.array_equal(host(ids)[t], rid), t
        near(host(lp)[t], [-np.log(2), -np.log(2), 0.0, 0.0][t], 8 * U, "logp")
        near(host(H)[t], [np.log(2), np.log(2), 0.0, 0.0][t], 8 * U, "entropy")
    d = host(svt.svt_token_logprobs_backward(dev(l), dev(np.array([1, V - 1, V - 1, V // 2])), nm, H, dev(np.ones(4, np.float32)),
                                             dev(np.ones(4, np.float32))))
    want = np.zeros((4, V))
    want[0, [1, V - 1]] = 0.5, -0.5
    want[1, [V - 1, 1]] = 0.5, -0.5
    near(d, want, 32 * U, "d_logits")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_embedding_backward_of_one_token_many_times(svt, kind):
    """All sums of one sign: n parts in float32 stay within the bound that n roundings would give, and far below."""
    say("one token", kind)
    for n, D in ((100000, 24), (4097, 130)):
        d = np.full((n, D), 0.7)
        dt = dev(d, ty(kind))
        one = float(host(dt)[0, 0])
        got = host(svt.svt_embedding_backward(dt, dev(np.full(n, 2)), 5, out_dtype=ty("f32")))
        # chains: 128 tokens at most in a chunk, then the chunks
        near(got[2], n * one, (128 + n / 8) * U * n * one, "sum")
        assert not got[[0, 1, 3, 4]].any()


# ---- sizes past 32 bits ------------------------------------------------------------------------------

def test_embedding_offsets_past_32_bits(svt):
    import torch
    say("large table")
    V, D = (1 << 21) + 77, 1032   # 2.2e9 elements
    table = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, 1 << 20, V - 2, V - 1], device="cuda")
    table[rows] = torch.randn((5, D), device="cuda").to(torch.bfloat16)
    ids = rows[torch.tensor([4, 0, 3, 1, 2, 4, 4], device="cuda")]
    assert torch.equal(svt.svt_embedding(table, ids), table[ids])
    del table
    d = torch.randn((7, D), device="cuda").to(torch.bfloat16)
    out = svt.svt_embedding_backward(d, ids, V, out_dtype=torch.float32)   # 8.7 GB of float32
    want = torch.zeros((5, D), dtype=torch.float64, device="cuda")
    for i, j in enumerate((4, 0, 3, 1, 2, 4, 4)):
        want[j] += d[i].double()
    assert torch.equal(out[rows[:4]].double(), want[:4])   # one part each
    assert ((out[V - 1].double() - want[4]).abs() <= 3 * U * sum(d[i].double().abs() for i in (0, 5, 6))).all()
    out[rows] = 0
    assert not any(out[i:i + (1 << 18)].any().item() for i in range(0, V, 1 << 18))


def test_logprobs_offsets_past_32_bits(svt):
    import torch
    say("many logits")
    T, V = 33000, 131075   # 4.3e9 elements
    logits = torch.empty((T, V), dtype=torch.bfloat16, device="cuda")
    base = torch.randn((8, V), device="cuda").to(torch.bfloat16)
    for i in range(0, T, 8):
        logits[i:i + 8] = base[:min(8, T - i)]
    tokens = torch.arange(T, device="cuda") % 8 * 1000
    lp, H, nm, ids, tlp = svt.svt_token_logprobs(logits, tokens, top=3)
    for a in (lp, H, nm, ids, tlp):   # T is a multiple of 8
        assert torch.equal(a.view(T // 8, 8, -1), a[:8].view(1, 8, -1).expand(T // 8, 8, -1))
    for t in range(8):
        r = S.Row(host(base)[t], 1.0)
        sums = U * (4 * r.away.max() + 3 * (65 + 10) + 8 * 65 + 16)   # 256 threads of 65 pieces of 8 values
        near(host(lp)[t], r.logp[1000 * t], sums + 40 * U * (1 + r.away.max()), "logp")
        near(host(H)[t], r.entropy, sums * (1 + 2 * r.spread) + 40 * U * (1 + r.spread), "entropy")
        assert np.array_equal(host(ids)[t], r.top(3)[0])
    one = torch.ones(T, device="cuda")
    want = svt.svt_token_logprobs_backward(base, tokens[:8], nm[:8], H[:8], one[:8], one[:8])
    svt.svt_token_logprobs_backward(logits, tokens, nm, H, one, one, out=(d := torch.empty_like(logits)))
    for i in range(0, T, 1000):
        assert torch.equal(d[i:i + 1000].view(-1, 8, V), want.view(1, 8, V).expand(125, 8, V))


def test_gated_offsets_past_32_bits(svt):
    """Rows, weights and the workspace of more than 2^32 bytes: their ends equal the same rows by themselves."""
    import torch
    say("many rows")
    R, K, N = 2300000, 1000, 24   # x 4.6 GB, dg and du
    x = torch.randn((R, K), device="cuda", dtype=torch.bfloat16)
    wg, wu = (torch.randn((N, K), device="cuda").to(torch.bfloat16) / 32 for _ in range(2))
    h, g, u = svt.svt_gated_linear(x, wg, wu, keep=True)
    tail = slice(R - 1000, R)
    f = svt.svt_gated_linear(x[tail].clone(), wg, wu, keep=True)
    for a, b in zip((h, g, u), f):
        assert torch.equal(a[tail], b)
    dh = torch.zeros((R, N), device="cuda", dtype=torch.bfloat16)
    dh[tail] = torch.randn((1000, N), device="cuda").to(torch.bfloat16)
    dx, dwg, dwu = svt.svt_gated_linear_backward(dh, x, wg, wu, g, u)
    want = svt.svt_gated_linear_backward(dh[tail].clone(), x[tail].clone(), wg, wu, *(t.clone() for t in f[1:]))
    assert not any(dx[i:i + 100000].any().item() for i in range(0, R - 1000, 100000) if i + 100000 <= R - 1000)
    # the sums may meet in another order: float32 sums of 2 N and of 1000 products, then one rounding.  A product is at most
    # the largest dh times the largest of 1.13 |u| and |g| (the slope, the value), times the largest weight or input
    far = float(dh.abs().max() * 1.13 * torch.maximum(f[1].abs().max(), f[2].abs().max()))
    for a, b, n, size in ((dx[tail], want[0], 2 * N, far * float(wg.abs().max())), (dwg, want[1], 1000, far * float(x[tail].abs().max())),
                          (dwu, want[2], 1000, far * float(x[tail].abs().max()))):
        a, b = a.double(), b.double()
        assert ((a - b).abs() <= 2 * HALF["bf16"] * b.abs() + 2 * sum_tol(n, n * size)).all()
        assert b.abs().max() > 20 * sum_tol(n, n * size)   # so that another row would show
    del x, dx, h, g, u, dh
    M, N, K = 512, 1100, 4000   # 4.5 GB each
    wg, wu = (torch.randn((M, N, K), device="cuda", dtype=torch.bfloat16) / 64 for _ in range(2))
    x = torch.randn((700, K), device="cuda").to(torch.bfloat16)
    for last in (3, 500):
        o = torch.zeros(M + 1, dtype=torch.int32, device="cuda")
        o[-2], o[-1] = 700 - last, 700     # expert 510: the first rows; 511: the last
        h, g, u = svt.svt_gated_linear(x, wg, wu, offsets=o, keep=True)
        for a, e in ((slice(0, 700 - last), 510), (slice(700 - last, 700), 511)):
            near(host(g[a]), host(x[a]) @ host(wg[e]).T,
                 sum_tol(K, np.abs(host(x[a])) @ np.abs(host(wg[e])).T) + HALF["bf16"] * np.abs(host(g[a])) * 1.01, "gate")
            near(host(u[a]), host(x[a]) @ host(wu[e]).T,
                 sum_tol(K, np.abs(host(x[a])) @ np.abs(host(wu[e])).T) + HALF["bf16"] * np.abs(host(u[a])) * 1.01, "up")
        dx, dwg, dwu = svt.svt_gated_linear_backward(h, x, wg, wu, g, u, offsets=o)
        for a, e in ((slice(0, 700 - last), 510), (slice(700 - last, 700), 511)):
            alone = svt.svt_gated_linear_backward(h[a].clone(), x[a].clone(), wg[e].clone(), wu[e].clone(), g[a].clone(), u[a].clone())
            far = float(h[a].abs().max() * 1.13 * torch.maximum(g[a].abs().max(), u[a].abs().max()))
            top_w, top_x, n = float(torch.maximum(wg[e].abs().max(), wu[e].abs().max())), float(x[a].abs().max()), a.stop - a.start
            for p, q, m, size in ((dx[a], alone[0], 2 * N, far * top_w), (dwg[e], alone[1], n, far * top_x),
                                  (dwu[e], alone[2], n, far * top_x)):
                p, q = p.double(), q.double()
                assert ((p - q).abs() <= 2 * HALF["bf16"] * q.abs() + 2 * sum_tol(m, m * size)).all()
        assert not dwg[:510].any() and not dwu[:510].any()


# ---- the largest sizes of one dimension ----------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_logprobs_of_the_longest_row(svt, kind):
    """2^30 tokens, equal but for three: log Z is known, and every token's gradient is one of four numbers.  A thread adds
    the 8 of a piece (8 u), then at most n = 2^30 / 8 / (256 threads) pieces' sums one after the other, each off by u of the sum
    so far: n u / 2 in all; then joins (16 u)."""
    import torch
    say("longest", kind)
    V = 1 << 30
    l = torch.zeros((1, V), dtype=ty(kind), device="cuda")
    places = [3, V // 2 + 1, V - 1]
    l[0, places] = torch.tensor([21.0, 20.0, 22.0], device="cuda").to(ty(kind))
    tokens = torch.tensor([V - 1], device="cuda")
    lp, H, nm, ids, tlp = svt.svt_token_logprobs(l, tokens, top=4)
    z = V - 3 + np.exp(21.0) + np.exp(20.0) + np.exp(22.0)
    p = np.exp([21.0, 20.0, 22.0, 0.0]) / z
    ent = -np.sum(p[:3] * np.log(p[:3])) - (V - 3) * p[3] * np.log(p[3])
    assert host(ids)[0].tolist() == [V - 1, 3, V // 2 + 1, 0]
    bound = (2.0 ** 19 / 2 + 24 + 30) * U   # 30: the exponentials and the logarithm
    near(host(lp)[0], np.log(p[2]), bound, "logp")
    near(host(H)[0], ent, bound * (1 + 2 * 22), "entropy")
    near(host(tlp)[0], np.log(p[[2, 0, 1, 3]]), bound, "alternatives")
    d = svt.svt_token_logprobs_backward(l, tokens, nm, H, torch.ones(1, device="cuda"))
    for i, w in ((3, -p[0]), (V // 2 + 1, -p[1]), (V - 1, 1 - p[2]), (0, -p[3]), (V - 2, -p[3])):
        near(np.float64(d[0, i].item()), w, (bound + 64 * U) * abs(p).max() + HALF[kind] * abs(w) + TINY[kind], f"d {i}")


@pytest.mark.parametrize("R, K, N", [(1, 1 << 20, 3), (70, 1 << 20, 3), (3, 5, 1 << 20), (70, 6, 1 << 20)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_gated_longest_sides(svt, R, K, N, kind):
    say("longest sides", R, K, N, kind)
    check(svt, R, K, N, None, "silu", kind, 0, "even")


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_embedding_of_the_widest_rows(svt, kind):
    import torch
    say("widest", kind)
    D = 1 << 24
    table = torch.randn((2, D), device="cuda").to(ty(kind))
    ids = torch.tensor([1, 2, 0, 1], device="cuda")
    out = svt.svt_embedding(table, ids)
    for i, v in enumerate((1, None, 0, 1)):
        assert torch.equal(out[i], table[v]) if v is not None else not out[i].any()
    d = svt.svt_embedding_backward(out, ids, 2)
    assert torch.equal(d[0], table[0]) and torch.equal(d[1], table[1] + table[1])


# ---- captured, on other streams, at once --------------------------------------------------------------

def every_call(svt, torch, kind, T, V, D, N, M):
    """(inputs, step): one call of every operator, over inputs that change in place."""
    z = lambda *s, dtype=ty(kind): torch.zeros(s, dtype=dtype, device="cuda")
    t = dict(table=z(V, D), ids=z(T, dtype=torch.int64), d=z(T, D), wg=z(M, N, D), wu=z(M, N, D), offsets=z(M + 1, dtype=torch.int32),
             logits=z(T, V), long=z(3, 50 * V), tok=z(3, dtype=torch.int64))

    def change():
        for name in ("table", "d", "wg", "wu", "logits", "long"):
            t[name].copy_(torch.randn(t[name].shape, device="cuda"))
        t["ids"].copy_(torch.randint(-1, V + 1, (T,), device="cuda"))
        t["tok"].copy_(torch.randint(0, 50 * V, (3,), device="cuda"))
        cuts = torch.randint(0, T + 1, (M + 1,), device="cuda").sort().values
        cuts[0], cuts[-1] = 0, T   # every row is an expert's, as outputs of the others would stay undefined
        t["offsets"].copy_(cuts)

    def step(stream=None):
        rows = svt.svt_embedding(t["table"], t["ids"], scale=1.5, stream=stream)
        dt = svt.svt_embedding_backward(t["d"], t["ids"], V, scale=0.5, stream=stream)
        dt2 = svt.svt_embedding_backward(t["d"], t["ids"], V, out=dt.clone(), accumulate=True, stream=stream) if stream is None else dt
        h, g, u = svt.svt_gated_linear(rows, t["wg"], t["wu"], offsets=t["offsets"], keep=True, stream=stream)
        dx, dwg, dwu = svt.svt_gated_linear_backward(h, rows, t["wg"], t["wu"], g, u, offsets=t["offsets"], stream=stream)
        one = svt.svt_gated_linear(rows[:1], t["wg"][0], t["wu"][0], activation="gelu", stream=stream)
        lp = svt.svt_token_logprobs(t["logits"], t["ids"], top=3, stream=stream)
        dl = svt.svt_token_logprobs_backward(t["logits"], t["ids"], lp[2], lp[1], lp[0], lp[1], stream=stream)
        few = svt.svt_token_logprobs(t["long"], t["tok"], top=5, stream=stream)
        return (rows, dt, dt2, h, g, u, dx, dwg, dwu, one, *lp, dl, *few)

    change()
    return change, step


SIZES = [("bf16", 900, 300, 64, 96, 4), ("f16", 9000, 2000, 33, 50, 9), ("f32", 700, 130, 40, 72, 3)]


@pytest.mark.parametrize("size", SIZES)
def test_captured_calls_replay(svt, size):
    """Two graphs, each with workspaces of its own: every replay, on inputs changed in place and with eager calls between,
    gives the eager bits, one after the other and both at once."""
    import torch
    say("graph", *size)
    graphs = []
    for _ in range(2):
        change, step = every_call(svt, torch, *size)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((change, step, g, got))
    streams = [torch.cuda.Stream() for _ in graphs]
    for i in range(4):
        wants = []
        for change, step, g, got in graphs:
            change()
            wants.append(step())
        torch.cuda.synchronize()
        for s, (_, _, g, _) in zip(streams, graphs):
            if i % 2:
                with torch.cuda.stream(s):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        for (_, _, _, got), want in zip(graphs, wants):
            for j, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), f"replay {i}, output {j}"


@pytest.mark.parametrize("size", SIZES)
def test_calls_on_other_streams_at_once(svt, size):
    import torch
    say("streams", *size)
    _, step = every_call(svt, torch, *size)
    torch.cuda.synchronize()
    want = step(torch.cuda.current_stream())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step(s))
    torch.cuda.synchronize()
    for g in got:
        for j, (a, b) in enumerate(zip(g, want)):
            assert torch.equal(a, b), j


# ---- together ----------------------------------------------------------------------------------------

class Scorer:
    """A token scorer: rows of a table, a routed net with a residual, logits against the same table."""

    def __init__(self, rng, V=23, D=12, N=20, E=4, K=2, T=14):
        self.V, self.D, self.N, self.E, self.K, self.T = V, D, N, E, K, T
        f = lambda *s: rng.normal(size=s).astype(np.float32)
        self.leaves = dict(table=f(V, D) / 2, router=f(D, E), wg=f(E, N, D) / 2, wu=f(E, N, D) / 2, down=f(E, D, N) / 3)
        self.ids, self.tokens = rng.integers(-1, V, T), rng.integers(0, V, T)
        self.dlp, self.dh = f(T), f(T) / 2
        self.scale, self.temper = 1.7, 0.8

    def loss(self, leaves):
        """(sum dlp logp + dh entropy, the choices) by the oracles."""
        x = S.embedding(leaves["table"], self.ids, self.scale)
        choice, w, _ = X.route(x @ leaves["router"], self.K, True)
        off, _, pos = X.sort(choice, self.E)
        rows = X.dispatch(x, pos, np.zeros((self.T * self.K, self.D)))
        h = S.gated(rows, leaves["wg"], leaves["wu"], "silu", off)[0]
        out = np.zeros_like(rows)
        for e in range(self.E):
            out[off[e]:off[e + 1]] = h[off[e]:off[e + 1]] @ leaves["down"][e].T
        y = x + X.combine(out, pos, w)[0]
        logits = y @ leaves["table"].T
        total = 0.0
        for t in range(self.T):
            r = S.Row(logits[t], self.temper)
            total += float(self.dlp[t]) * r.logp[self.tokens[t]] + float(self.dh[t]) * r.entropy   # all in 64 bits
        return total, choice

    def run(self, svt, torch, dtype):
        """The loss and every leaf's gradient on the GPU."""
        L = {k: dev(v).to(dtype) for k, v in self.leaves.items()}
        ids, tokens = dev(self.ids), dev(self.tokens)
        x = svt.svt_embedding(L["table"], ids, scale=self.scale)
        l = x @ L["router"]
        choice, w = svt.svt_route(l, self.K)
        off, order, pos = svt.svt_expert_sort(choice, self.E)
        rows = svt.svt_expert_dispatch(x, pos)
        h, g, u = svt.svt_gated_linear(rows, L["wg"], L["wu"], offsets=off, keep=True)
        ends = off.tolist()
        parts = [slice(a, b) for a, b in zip(ends, ends[1:])]
        out = torch.cat([h[p] @ L["down"][e].t() for e, p in enumerate(parts)])
        y = x + svt.svt_expert_combine(out, pos, w)
        logits = (y @ L["table"].t()).contiguous()
        lp, H, norms = svt.svt_token_logprobs(logits, tokens, scale=self.temper)
        d_lp, d_h = dev(self.dlp), dev(self.dh)
        dl = svt.svt_token_logprobs_backward(logits, tokens, norms, H, d_lp, d_h, scale=self.temper)
        dy = (dl @ L["table"]).contiguous()
        d_table = (dl.t() @ y).contiguous()
        d_out, d_w = svt.svt_expert_combine_backward(dy, out, pos, w)
        d_down = torch.stack([d_out[p].t() @ h[p] for p in parts])
        d_hid = torch.cat([d_out[p] @ L["down"][e] for e, p in enumerate(parts)])
        d_rows, d_wg, d_wu = svt.svt_gated_linear_backward(d_hid, rows, L["wg"], L["wu"], g, u, offsets=off)
        d_l = svt.svt_route_backward(l, choice, w, d_w)
        d_x = dy + svt.svt_expert_dispatch_backward(d_rows, pos) + d_l @ L["router"].t()
        d_table = svt.svt_embedding_backward(d_x.contiguous(), ids, self.V, scale=self.scale, out=d_table, accumulate=True)
        loss = float((d_lp.double() * lp.double() + d_h.double() * H.double()).sum())
        return loss, dict(table=d_table, router=x.t() @ d_l, wg=d_wg, wu=d_wu, down=d_down)


def test_training_step_of_a_scorer(svt):
    """The operators in the order of a training step, with the router and the exchange: the loss and every leaf's gradient
    against differences of the float64 oracles.  A value passes some 12 steps, each a float32 sum of at most 40 terms, so
    500 roundings at most, relative to magnitudes that stay below 16 times the largest gradient: 5e-4 of it; differences
    are good to h^2."""
    import torch
    say("training step")
    m = Scorer(np.random.default_rng(8))
    loss, grads = m.run(svt, torch, torch.float32)
    leaves = {k: v.astype(np.float64) for k, v in m.leaves.items()}
    want, choice = m.loss(leaves)
    assert abs(loss - want) < 1e-4 * (1 + abs(want))
    h = 1e-5
    for name, a in leaves.items():
        got = host(grads[name])
        d = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep, f = a[i], []
            for s in (h, -h):
                a[i] = keep + s
                v, now = m.loss(leaves)
                assert np.array_equal(now, choice)
                f.append(v)
            a[i] = keep
            d[i] = (f[0] - f[1]) / (2 * h)
        assert np.abs(d).max() > 0.1, name   # a gradient there is
        near(got, d, 5e-4 * np.abs(d).max() + 1e-7, name)


def test_found_candidates_are_scored(svt):
    """The candidates of a search (padded with -1) as tokens: rows of their table, gated products, log probabilities of the
    best and a next token's alternatives, one query at a time as serving does and all at once: the same bits by row."""
    import oracle_pins as P
    import torch
    say("search to scores")
    rng = np.random.default_rng(4)
    items, sigs, cl, cent = P.small_catalogue(rng, n=3000, d=64, nlist=8, W=2)
    ix = svt.Index(items, sigs, cl, cent, 1.0)
    q = rng.integers(-127, 128, (3, 64)).astype(np.int8)
    ids, *_ = ix.search(dev(q), dev(np.zeros((3, 2), np.int64)), 4, 60)
    tokens = ids.to(torch.int64)
    table = dev(rng.normal(size=(3000, 48)), ty("bf16"))
    wg, wu = (dev(rng.normal(size=(80, 48)) / 7, ty("bf16")) for _ in range(2))
    head = dev(rng.normal(size=(80, 500)) / 9, torch.float32)
    x = svt.svt_embedding(table, tokens.reshape(-1))
    c = host(tokens).reshape(-1)
    assert np.array_equal(host(x), S.embedding(host(table), c, 1.0))
    h = svt.svt_gated_linear(x, wg, wu)
    rh, rg, ru, sg, su = S.gated(host(x), host(wg)[None], host(wu)[None], "silu")
    tg, tu = sum_tol(48, sg), sum_tol(48, su)
    value = S.activation(rg, "silu")[0]
    th = (np.abs(ru) + tu) * (1.13 * tg + act_tol(rg) * np.abs(value)) + np.abs(value) * tu + U * np.abs(rh)
    near(host(h), rh, th + HALF["bf16"] * (np.abs(rh) + th) + TINY["bf16"], "h")
    logits = (h.float().view(3, 60, 80).mean(1) @ head).contiguous()
    every = svt.svt_token_logprobs(logits, tokens[:, 0] % 500, top=5)
    for b in range(3):
        one = svt.svt_token_logprobs(logits[b:b + 1].clone(), (tokens[b:b + 1, 0] % 500).contiguous(), top=5)
        assert np.array_equal(host(one[3]), host(every[3])[b:b + 1])
        r = S.Row(host(logits)[b], 1.0)
        assert np.array_equal(host(every[3])[b], r.top(5)[0])
        near(host(one[4])[0], r.top(5)[1], 100 * U * (1 + r.away.max()), "alternatives")
    ix.close()
