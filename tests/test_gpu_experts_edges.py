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


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [11, 64, 300])
def test_route_weights_below_the_smallest_normal_float(svt, E, renorm, kind):
    """Experts 80 to 110 below the best: weights down to the smallest subnormal, and their gradients.  The exponential
    and the division each round a subnormal by at most 2^-150; the gradient's two products by as much, and pass the
    first on by |dw| + |dot|."""
    say("subnormal", E, renorm, kind)
    rng = np.random.default_rng(E)
    gaps = np.array([0, 80, 87, 87.4, 88, 92, 95, 100, 103, 103.9, 110])
    l = np.full((6, E), -np.inf)
    for t in range(6):
        l[t, rng.permutation(E)[:11]] = rng.normal() - gaps - 0.1 * rng.random(11)
    lt = dev(l, ty(kind))
    l = host(lt)
    for K in (8, 11):
        ids, w = svt.svt_route(lt, K, renormalise=renorm)
        rid, rw, sens = X.route(l, K, renorm)
        assert np.array_equal(host(ids), rid)
        near(host(w), rw, U * rw * (sens + 31) + 2.0 ** -149, "weights")
        dw = rng.normal(size=(6, K)).astype(np.float32)
        d = svt.svt_route_backward(lt, ids, w, dev(dw), renormalise=renorm, out=dev(np.zeros((6, E)), ty(kind)))
        rd, mag, bs = X.route_backward(l, rid, host(w), dw.astype(np.float64), renorm)
        most = np.abs(dw).max(1, keepdims=True).astype(np.float64)
        near(host(d), rd, U * mag * (bs + 51) + HALF[kind] * np.abs(rd) + TINY[kind] + 2.0 ** -149 * (2 * most + 1),
             "d_logits")


@pytest.mark.parametrize("E", [8, 16, 64, 512])
@pytest.mark.parametrize("K", [3, 8])
def test_route_backward_adds_a_repeated_expert_in_order(svt, E, K):
    """An expert that a token names several times gets the sum of its parts in the order of the choices, whatever
    lanes hold them.  Parts of 32 binades, so that the float32 sum depends on the order; weights of 0, so that the
    parts are dw; equal logits, so that p is the power of two 1 / E: the result is that sum, exactly."""
    say("repeated", E, K)
    rng = np.random.default_rng(E + K)
    T = 300
    ids = np.stack([rng.choice(rng.choice(E, 2, replace=False), K) for _ in range(T)]).astype(np.int32)
    dw = rng.choice([1.0, -1.0], (T, K)) * rng.uniform(1, 2, (T, K)) * 2.0 ** rng.integers(-4, 28, (T, K))
    dw = dw.astype(np.float32)
    want = np.zeros((T, E), np.float32)
    for t in range(T):
        for j in range(K):
            want[t, ids[t, j]] += dw[t, j]
    want *= np.float32(1.0 / E)
    for _ in range(3):
        got = svt.svt_route_backward(dev(np.zeros((T, E), np.float32)), dev(ids), dev(np.zeros((T, K), np.float32)),
                                     dev(dw), renormalise=False)
        assert np.array_equal(host(got).astype(np.float32), want)


# ---- exchange ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [1 << 22, (1 << 22) + 4, 3000001])
def test_combine_backward_of_wide_rows(svt, D, kind):
    """d_weights of wide rows, constant (every addition rounds the same way) and random.  A lane has m = ceil(pieces /
    64) pieces of n values (16 bytes, or what divides the row): n products in a chain, up to 512 pieces' sums, ceil(m
    / 512) sums of those, 6 levels across lanes: (n + min(m, 512) + ceil(m / 512) + 6) u of sum |dy r|."""
    say("wide", D, kind)
    import torch
    size = 4 if kind == "f32" else 2
    v = next(b for b in (16, 8, 4, 2) if D * size % b == 0)
    n, m = v // size, -(-(D * size // v) // 64)
    bound = (n + min(m, 512) + -(-m // 512) + 6) * U
    g = torch.Generator(device="cuda").manual_seed(D)
    dy = torch.randn((2, D), generator=g, device="cuda").to(ty(kind))
    rows = torch.randn((4, D), generator=g, device="cuda").to(ty(kind))
    dy[0], rows[0], rows[1] = 0.7, 1.1, 0.1
    pos = torch.tensor([[0, 1], [3, 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 2.0], [1.0, -1.0]], device="cuda")
    dr, dw = svt.svt_expert_combine_backward(dy, rows, pos, w)
    for t in range(2):
        for j in range(2):
            a, b = dy[t].double(), rows[int(pos[t, j])].double()
            near(np.float64(dw[t, j].item()), float(a @ b), bound * float(a.abs() @ b.abs()), f"d_weights {t} {j}")
            assert torch.equal(dr[int(pos[t, j])], (w[t, j] * dy[t].float()).to(ty(kind)))


# ---- 4-bit products with float32 outputs ---------------------------------------------------------------

def pack(svt, q, s, z, K, G, scale_kind="f32"):
    q = np.pad(q, ((0, 0), (0, 0), (0, K % 2)))
    return svt.svt_quant_pack(dev(q[..., 0::2] | (q[..., 1::2] << 4)), dev(s, ty(scale_kind)), None if z is None else dev(z),
                              K, G)


# rows, outputs, inputs, group; rows of each expert instead of one number: products by expert
PRECISE = [(1, 300, 1030, 128), (16, 2048, 4096, 64), (16, 16400, 1100, 128), (40, 2100, 1030, 32), (9, 700, 1500, 128),
           (64, 8200, 260, 64), (520, 4100, 261, 128), (1030, 4100, 260, 64), (1030, 4100, 130, 32),
           ([200, 90, 33, 0, 250, 1, 140, 61], 4100, 261, 128), ([3] * 30 + [0, 50], 1500, 389, 64), ([1, 0, 2, 5], 40, 1030, 32)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("R, N, K, G", PRECISE)
def test_float32_outputs_lose_nothing_to_zero_points(svt, R, N, K, G, zeros, kind):
    """Rows behind a relu (no negative value) times weights most of which are 0, that is q at its zero point: errors
    stay in proportion to sum |s| |x| |q - z|, and outputs whose weights are all 0 are the bias itself.  n = parts G +
    groups + 12 roundings of independent sign: 4 sqrt(n) u, as for every product; q - z itself is exact."""
    say("precise", R, N, K, G, zeros, kind)
    counts = R if isinstance(R, list) else [R]
    M, off = len(counts), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rng = np.random.default_rng(N + K + G)
    groups = -(-K // G)
    z = rng.integers(0, 16, (M, N, groups)).astype(np.uint8) if zeros else None
    zk = np.repeat(np.full((M, N, groups), 8, np.uint8) if z is None else z, G, 2)[:, :, :K]
    q = np.where(rng.random((M, N, K)) < 1 / 128, rng.integers(0, 16, (M, N, K)), zk).astype(np.uint8)
    q[:, ::7] = zk[:, ::7]
    s = rng.normal(size=(M, N, groups)).astype(np.float32)
    x = dev(np.maximum(rng.normal(size=(off[-1], K)) + 0.5, 0), ty(kind))
    bias = rng.normal(size=(M, N)).astype(np.float32)
    y = host(svt.svt_quant_linear(x, pack(svt, q, s, z, K, G), offsets=dev(off) if M > 1 else None, bias=dev(bias),
                                  out_dtype=ty("f32")))
    hx, n = host(x), (3 if kind == "f32" else 1) * G + groups + 12
    for e in range(M):
        rows, w = hx[off[e]:off[e + 1]], np.repeat(s[e].astype(np.float64), G, 1)[:, :K] * (q[e].astype(np.float64) - zk[e])
        want, mag = rows @ w.T + bias[e], np.abs(rows) @ np.abs(w).T + np.abs(bias[e])
        near(y[off[e]:off[e + 1]], want, 4 * np.sqrt(n) * U * mag + U * np.abs(want), f"expert {e}")
        assert np.all(y[off[e]:off[e + 1], ::7] == bias[e, ::7])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_any_zero_point_is_exact(svt, G, kind):
    """Zero points are whole bytes: rows of the identity return s (q - z), rounded once, up to z = 255."""
    rng = np.random.default_rng(G + 1)
    K, N = 260, 48
    groups = -(-K // G)
    q = rng.integers(0, 16, (1, N, K)).astype(np.uint8)
    z = rng.choice([0, 1, 15, 16, 127, 128, 200, 254, 255], (1, N, groups)).astype(np.uint8)
    s = rng.normal(size=(1, N, groups)).astype(np.float32)
    y = svt.svt_quant_linear(dev(np.eye(K), ty(kind)), pack(svt, q, s, z, K, G), out_dtype=ty("f32"))
    want = np.repeat(s[0], G, 1)[:, :K] * (q[0].astype(np.float32) - np.repeat(z[0], G, 1)[:, :K].astype(np.float32))
    assert np.array_equal(host(y).astype(np.float32), want.T)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("R, N, K, G", [(1, 40, 197, 64), (9, 70, 5, 32), (40, 2100, 1030, 128), (600, 4100, 203, 32)])
def test_float32_outputs_of_rows_with_infinities(svt, R, N, K, G, zeros, kind):
    """A row that holds an infinity or NaN gets NaN outputs in every form, wherever it lies (in a row's last, short piece
    too); the largest finite values do not, and other rows keep their bits."""
    say("infinities", R, N, K, G, zeros, kind)
    rng = np.random.default_rng(R + K)
    groups = -(-K // G)
    q = rng.integers(0, 16, (1, N, K)).astype(np.uint8)
    z = rng.integers(0, 256, (1, N, groups)).astype(np.uint8) if zeros else None
    w = pack(svt, q, 0.125 * rng.normal(size=(1, N, groups)).astype(np.float32), z, K, G)
    most = {"f32": 2.0 ** 100, "f16": 65504.0, "bf16": 2.0 ** 100}[kind]   # sums stay finite
    x = rng.normal(size=(R, K))
    x[::3, 0] = most
    clean = host(svt.svt_quant_linear(dev(x, ty(kind)), w, out_dtype=ty("f32")))
    assert np.all(np.isfinite(clean))
    for value in (np.inf, -np.inf, np.nan):
        for at in {0, K // 2, K - 1}:
            bad = x.copy()
            bad[R // 2, at] = value
            y = host(svt.svt_quant_linear(dev(bad, ty(kind)), w, out_dtype=ty("f32")))
            assert np.all(np.isnan(y[R // 2]))
            others = np.arange(R) != R // 2
            assert np.array_equal(y[others], clean[others])


# ---- tensors that require grad -------------------------------------------------------------------------

def test_history_is_refused_or_not_wanted(svt):
    """Every floating argument that requires grad is refused in grad mode, outputs too; under no_grad it is not."""
    import torch
    rng = np.random.default_rng(0)
    T, E, K, D = 5, 8, 2, 64
    x, l, dy = [dev(rng.normal(size=s).astype(np.float32)) for s in ((T, D), (T, E), (T, D))]
    ids, w = svt.svt_route(l, K)
    off, order, pos = svt.svt_expert_sort(ids, E)
    rows = svt.svt_expert_dispatch(x, pos)
    bias, s = dev(np.zeros((E, 16), np.float32)), dev(np.ones((E, 16, 2), np.float32))
    nib = dev(rng.integers(0, 256, (E, 16, 32)).astype(np.uint8))
    packed = svt.svt_quant_pack(nib, s, None, D, 32)
    calls = [(l, lambda g: svt.svt_route(g, K)), (l, lambda g: svt.svt_route_backward(g, ids, w, w)),
             (w, lambda g: svt.svt_route(l, K, out_weights=g)),
             (w, lambda g: svt.svt_route_backward(l, ids, g, w)), (w, lambda g: svt.svt_route_backward(l, ids, w, g)),
             (x, lambda g: svt.svt_expert_dispatch(g, pos)), (rows, lambda g: svt.svt_expert_dispatch(x, pos, out=g)),
             (rows, lambda g: svt.svt_expert_dispatch_backward(g, pos)), (rows, lambda g: svt.svt_expert_combine(g, pos, w)),
             (w, lambda g: svt.svt_expert_combine(rows, pos, g)),
             (dy, lambda g: svt.svt_expert_combine_backward(g, rows, pos, w)),
             (rows, lambda g: svt.svt_expert_combine_backward(dy, g, pos, w)),
             (w, lambda g: svt.svt_expert_combine_backward(dy, rows, pos, g)),
             (s, lambda g: svt.svt_quant_pack(nib, g, None, D, 32)),
             (rows, lambda g: svt.svt_quant_linear(g, packed, offsets=off)),
             (bias, lambda g: svt.svt_quant_linear(rows, packed, offsets=off, bias=g))]
    for t, call in calls:
        g = t.clone().requires_grad_()
        with pytest.raises(ValueError, match="requires grad"):
            call(g)
        with torch.no_grad():
            call(g)


def test_combine_in_an_autograd_function(svt):
    """As a training program uses the calls: inside an autograd function, where torch records nothing."""
    import torch

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, pos, w):
            ctx.save_for_backward(rows, pos, w)
            return svt.svt_expert_combine(rows, pos, w)

        @staticmethod
        def backward(ctx, dy):
            rows, pos, w = ctx.saved_tensors
            dr, dw = svt.svt_expert_combine_backward(dy.contiguous(), rows, pos, w)
            return dr, None, dw

    rng = np.random.default_rng(1)
    rows = dev(rng.normal(size=(6, 10)).astype(np.float32)).requires_grad_()
    w = dev(rng.normal(size=(3, 2)).astype(np.float32)).requires_grad_()
    pos = dev(np.array([[5, 0], [1, 2], [4, 3]], np.int32))
    dy = dev(rng.normal(size=(3, 10)).astype(np.float32))
    Combine.apply(rows, pos, w).backward(dy)
    want_rows, want_w = torch.zeros(6, 10, device="cuda"), torch.zeros(3, 2, device="cuda")
    for t in range(3):
        for j in range(2):
            want_rows[int(pos[t, j])] = w.detach()[t, j] * dy[t]
            want_w[t, j] = (dy[t].double() * rows.detach()[int(pos[t, j])].double()).sum()
    assert torch.equal(rows.grad, want_rows)
    near(host(w.grad), host(want_w), 17 * U * 10 * 16, "d_weights")   # 10 products of values below 4


# ---- ends of the ranges that nothing else reaches --------------------------------------------------------

@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_route_backward_of_infinite_logits(svt, renorm, kind):
    """One and two logits of +inf: the gradient of a finite peak (the oracle's), no NaN."""
    l = np.zeros((3, 10))
    l[0, 3], l[1, [2, 7]], l[2, [0, 9]] = np.inf, np.inf, (np.inf, 5.0)
    l[2, 4] = -np.inf
    lt = dev(l, ty(kind))
    ids, w = svt.svt_route(lt, 4, renormalise=renorm)
    rid, rw, _ = X.route(l, 4, renorm)
    assert np.array_equal(host(ids), rid) and np.array_equal(host(w), rw)   # 0, 1/2 and 1
    dw = np.random.default_rng(3).normal(size=(3, 4)).astype(np.float32)
    d = svt.svt_route_backward(lt, ids, w, dev(dw), renormalise=renorm)
    rd, mag, _ = X.route_backward(l, rid, rw, dw.astype(np.float64), renorm)
    near(host(d), rd, U * mag * 51 + HALF[kind] * np.abs(rd) + TINY[kind], "d_logits")


def test_exchange_more_tokens_than_one_grid(svt):
    """4.3 M tokens of 33 bfloat16 (2-byte pieces, a wave per token): workgroups go round a second time from token
    4194304 on.  One choice per token, so every result but d_weights is one product, rounded once in float32 and
    once to the type; a d_weight is 33 products in 64 lanes: one product, two sums of one, 6 levels."""
    import torch
    T, D = 4300003, 33
    g = torch.Generator(device="cuda").manual_seed(1)
    pos = torch.randperm(T, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    at = pos[:, 0].long()
    x = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    rows = svt.svt_expert_dispatch(x, pos)
    assert torch.equal(rows[at], x)
    assert torch.equal(svt.svt_expert_dispatch_backward(rows, pos), x)
    w = torch.randn((T, 1), generator=g, device="cuda")
    assert torch.equal(svt.svt_expert_combine(rows, pos, w), (w * x.float()).bfloat16())
    dy = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    dr, dw = svt.svt_expert_combine_backward(dy, rows, pos, w)
    assert torch.equal(dr[at], (w * dy.float()).bfloat16())
    want = (dy.double() * x.double()).sum(1, keepdim=True)
    mag = (dy.double() * x.double()).abs().sum(1, keepdim=True)
    assert bool(((dw.double() - want).abs() <= 9 * U * mag).all())


@pytest.mark.parametrize("kind, least", [("bf16", -133), ("f16", -24), ("f32", -133)])
@pytest.mark.parametrize("R, N", [(1, 40), (40, 48), (200, 4200)])
def test_linear_subnormal_rows(svt, R, N, kind, least):
    """Rows of the types' smallest values, subnormals among them, one value per row: whole multiples of 2^least times q
    - 8, exactly.  (float32 rows: digits below 2^-133 are not used.)"""
    rng = np.random.default_rng(R)
    K = 70
    q = rng.integers(0, 16, (1, N, K)).astype(np.uint8)
    x, at = np.zeros((R, K)), rng.integers(0, K, R)
    whole = rng.integers(1, 2 ** (20 if kind == "f32" else 8), R)
    x[np.arange(R), at] = rng.choice([-1, 1], R) * whole * 2.0 ** least
    xt = dev(x, ty(kind))
    assert np.array_equal(host(xt), x)
    y = svt.svt_quant_linear(xt, pack(svt, q, np.ones((1, N, 3), np.float32), None, K, 32), out_dtype=ty("f32"))
    near(host(y), x @ (q[0].astype(np.float64) - 8).T, 0.0, "subnormal")
    if kind == "f32":   # what lies below the used digits adds less than one of them
        fine = (x + np.where(x != 0, np.sign(x) * 2.0 ** -134, 0)).astype(np.float32)
        y = svt.svt_quant_linear(dev(fine), pack(svt, q, np.ones((1, N, 3), np.float32), None, K, 32))
        near(host(y), fine.astype(np.float64) @ (q[0].astype(np.float64) - 8).T, 8 * 2.0 ** -133, "subnormal")
