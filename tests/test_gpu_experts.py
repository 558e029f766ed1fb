"""Routed-expert operators on the GPU against the float64 oracle (oracle/experts.py).

Integers (experts, order, positions, offsets) and copied rows are equal.  Numbers stay within bounds that are
derived from the kernels' float32 arithmetic, u = 2^-24 (half a step, relative):
  route     a weight is e_s / sum e with e = exp(l - max): the difference is rounded (u |l - max| relative in
            e), expf is off by at most 2 ulp (4 u), the sum adds at most 512 terms in chains of at most 16 and
            6 levels (22 u), the division 1 u.  Relative: u (|l_s - max| + sum p |l - max| + 4 + 4 + 22 + 1).
            The middle terms are the oracle's sensitivity.  Float underflow adds 2^-126.
  gradient  d = p (g - dot): p as above, the sums over at most 16 choices and the products at most 20 u of
            p (|g| + sum |dw w|); then one rounding to the type.
  combine   a chain of top products and sums in float32: top u sum |w r|, then one rounding.
  d_rows    one product (u) and one rounding.  d_weights: at most ceil(D / lanes) products in a chain, then 6
            levels: u (D / 64 + 8 + 8) sum |dy r|, since a lane holds at most 8 neighbouring values more.
  linear    products x q are exact.  Group sums add G (x 3 parts for float32) terms, then the zero-point term,
            the scales and the sums over groups and waves: n = parts G + groups + 12 roundings.  Rounding
            errors of independent sign grow like their root: 4 sqrt(n) u (Higham and Mary's probabilistic
            bound with lambda = 4) of A = sum |s| |x| (q + z) + |b|; then one rounding.
A rounding to a type is off by eps / 2 relative, or half the smallest subnormal."""
import ctypes

import numpy as np
import pytest

from gpu_common import say
from oracle import experts as X

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


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
    assert out.is_contiguous()
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


# ---- router ------------------------------------------------------------------------------------------

ROUTES = [(1, 1, 1), (1, 8, 2), (3, 7, 7), (65, 9, 4), (64, 16, 16), (33, 31, 5), (130, 64, 8), (17, 100, 3),
          (9, 128, 8), (40, 255, 16), (12, 256, 1), (5, 511, 16), (6, 512, 16),
          (7, 512, 8), (3, 257, 7), (21, 250, 8), (5, 12, 12), (9, 30, 10), (33, 60, 9), (4, 120, 13), (600, 16, 8)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T, E, K", ROUTES)
def test_route_and_backward(svt, T, E, K, renorm, kind):
    say("route", T, E, K, renorm, kind)
    rng = np.random.default_rng(T * 1000 + E + K)
    l = 2.0 * rng.normal(size=(T, E))
    shut = rng.random((T, E)) < 0.15
    l[shut] = np.where(rng.random(int(shut.sum())) < 0.5, -np.inf, np.nan)
    if T > 2:
        l[1] = -np.inf                      # nothing open
        l[2] = 0.25                         # every expert tied
    lt = dev(l, ty(kind), shift=1)
    l = host(lt)
    ids, w = svt.svt_route(lt, K, renormalise=renorm)
    rid, rw, sens = X.route(l, K, renorm)
    assert np.array_equal(host(ids), rid)
    near(host(w), rw, U * rw * (sens + 31) + 2.0 ** -126, "weights")
    dw = rng.normal(size=(T, K)).astype(np.float32)
    d = svt.svt_route_backward(lt, ids, w, dev(dw), renormalise=renorm)
    rd, mag, bsens = X.route_backward(l, rid, host(w), dw.astype(np.float64), renorm)
    near(host(d), rd, U * mag * (bsens + 31 + 20) + HALF[kind] * np.abs(rd) + TINY[kind] + 2.0 ** -126, "d_logits")


def test_route_more_tokens_than_one_grid(svt):
    """270,000 tokens of 512 experts: workgroups go round more than once; tokens of every part are compared."""
    import torch
    T, E, K = 270000, 512, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    l = torch.randn((T, E), generator=g, device="cuda").bfloat16()
    ids, w = svt.svt_route(l, K)
    dw = torch.randn((T, K), generator=g, device="cuda")
    d = svt.svt_route_backward(l, ids, w, dw)
    pick = [0, 1, 3, 4, 131071, 262139, 262143, 262144, 262145, 269998, 269999]
    rl = host(l[pick])
    rid, rw, sens = X.route(rl, K, True)
    assert np.array_equal(host(ids[pick]), rid)
    near(host(w[pick]), rw, U * rw * (sens + 31) + 2.0 ** -126, "weights")
    rd, mag, bs = X.route_backward(rl, rid, host(w[pick]), host(dw[pick]), True)
    near(host(d[pick]), rd, U * mag * (bs + 51) + HALF["bf16"] * np.abs(rd) + TINY["bf16"], "d_logits")


def test_route_infinite_logits(svt):
    l = np.array([[np.inf, 0.0, np.inf, -1.0], [3e38, -3e38, np.inf, 1.0]], np.float32)
    ids, w = svt.svt_route(dev(l), 3)
    assert host(ids).tolist() == [[0, 2, 1], [2, 0, 3]]
    assert host(w).tolist() == [[0.5, 0.5, 0.0], [1.0, 0.0, 0.0]]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_route_zeros_tie_and_neighbours_do_not(svt, kind):
    """-0 ties with 0 (the lower expert first); logits one step of the type apart do not."""
    step = 1.0 + 2 * HALF[kind]
    l = np.array([[0.0, -0.0, 0.0, -0.0, -1.0, 0.0], [1.0, step, 1.0, -step, -1.0, step]])
    ids, _ = svt.svt_route(dev(l, ty(kind)), 6)
    assert host(ids).tolist() == [[0, 1, 2, 3, 5, 4], [1, 5, 0, 2, 4, 3]]
    ids, _ = svt.svt_route(dev(l[:, ::-1].copy(), ty(kind)), 6)
    assert host(ids).tolist() == [[0, 2, 3, 4, 5, 1], [0, 4, 3, 5, 1, 2]]


def test_route_backward_ignores_foreign_experts(svt):
    l = dev(np.zeros((1, 4), np.float32))
    ids = dev(np.array([[-1, 9, 2, -2 ** 31]], np.int32))
    ones = dev(np.ones((1, 4), np.float32))
    assert host(svt.svt_route_backward(l, ids, ones, ones, renormalise=True)).tolist() == [[0, 0, 0, 0]]
    twice = dev(np.array([[2, 2, 0, 2]], np.int32))   # an expert named more than once gets every part
    half = dev(np.full((1, 4), 0.5, np.float32))
    got = svt.svt_route_backward(l, twice, half, dev(np.array([[1.0, 2.0, 4.0, 8.0]], np.float32)), renormalise=True)
    assert host(got).tolist() == [[0.5 * (4 - 7.5), 0, 0.5 * (11 - 3 * 7.5), 0]]
    w = dev(np.full((1, 4), 0.25, np.float32))
    assert host(svt.svt_route_backward(l, ids, w, ones, renormalise=False)).tolist() == [[-0.0625, -0.0625, 0.1875, -0.0625]]


# ---- sort --------------------------------------------------------------------------------------------

SORTS = [(0, 1, 4), (1, 1, 1), (1, 16, 512), (64, 4, 32), (63, 3, 5), (1000, 2, 8), (4097, 1, 1), (8192, 2, 64),
         (8193, 2, 64), (5462, 3, 300), (40000, 1, 512), (70001, 3, 17), (30000, 16, 128), (1 << 20, 3, 64)]


@pytest.mark.parametrize("T, K, E", SORTS)
@pytest.mark.parametrize("mode", ["spread", "one", "dropped", "all_dropped"])
def test_sort(svt, T, K, E, mode):
    say("sort", T, K, E, mode)
    rng = np.random.default_rng(T + K + E)
    e = rng.integers(0, E, (T, K)) if mode != "one" else np.full((T, K), E - 1)
    if mode == "dropped":
        e = np.where(rng.random((T, K)) < 0.3, rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1], (T, K)), e)
    if mode == "all_dropped":
        e = np.full((T, K), -1)
    e = e.astype(np.int32)
    off, order, pos = [host(t) for t in svt.svt_expert_sort(dev(e), E)]
    flat = e.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    want = np.argsort(key, kind="stable").astype(np.int32)
    n = int((key < E).sum())
    if T * K <= 5000:
        ro, rr, rp = X.sort(e, E)
        assert np.array_equal(off, ro) and np.array_equal(order, rr) and np.array_equal(pos, rp)
    assert np.array_equal(off, np.searchsorted(key[want], np.arange(E + 1)))
    assert np.array_equal(order[:n], want[:n]) and np.all(order[n:] == -1)
    place = np.full(T * K, -1, np.int32)
    place[want[:n]] = np.arange(n)
    assert np.array_equal(pos.reshape(-1), place)


def test_sort_dirty_workspace_and_small_one(svt):
    import torch
    e = dev(np.random.default_rng(5).integers(0, 9, (30000, 2)).astype(np.int32))
    need = svt.svt_expert_sort_workspace_size(30000, 2, 9)
    a = svt.svt_expert_sort(e, 9)
    b = svt.svt_expert_sort(e, 9, workspace=torch.full((need,), 0xAB, dtype=torch.uint8, device="cuda"))
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    with pytest.raises(svt.SvtError, match="workspace"):
        svt.svt_expert_sort(e, 9, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


# ---- exchange ----------------------------------------------------------------------------------------

EXCHANGES = [(1, 1, 1, 1), (1, 2, 64, 4), (5, 3, 7, 2), (33, 2, 250, 8), (17, 4, 129, 5), (64, 6, 96, 16),
             (40, 5, 1000, 8), (9, 16, 520, 20), (300, 1, 128, 3), (7, 2, 4100, 4)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("T, K, D, E", EXCHANGES)
def test_exchange(svt, T, K, D, E, shift, kind):
    say("exchange", T, K, D, E, shift, kind)
    import torch
    rng = np.random.default_rng(T + K + D)
    e = rng.integers(0, E, (T, K)).astype(np.int32)
    e[rng.random((T, K)) < 0.2] = -1
    if T > 3:
        e[3] = -1
    off, order, pos = svt.svt_expert_sort(dev(e), E)
    p, n = host(pos), int(host(off)[-1])
    x, rows, dy = [dev(rng.normal(size=s), ty(kind), shift) for s in ((T, D), (T * K, D), (T, D))]
    rows[n:] = float("nan")                       # rows that no entry names are not read
    w = rng.normal(size=(T, K)).astype(np.float32)
    wd = dev(w)
    mark = lambda *s: dev(np.full(s, 7.0), ty(kind), shift)

    sent = svt.svt_expert_dispatch(x, pos, out=mark(T * K, D))
    want = X.dispatch(host(x), p, np.full((T * K, D), 7.0))
    assert np.array_equal(host(sent), want)

    def rounding(v):
        return HALF[kind] * np.abs(v) + TINY[kind]

    hr = np.nan_to_num(host(rows))
    for weights in (w, None):
        y = svt.svt_expert_combine(rows, pos, None if weights is None else wd, out=mark(T, D))
        ry, mag = X.combine(hr, p, weights)
        near(host(y), ry, K * U * mag * (1 + 2 * HALF[kind]) + rounding(ry), "combine")
    dx = svt.svt_expert_dispatch_backward(rows, pos, out=mark(T, D))
    ry, mag = X.combine(hr, p, None)
    near(host(dx), ry, K * U * mag * (1 + 2 * HALF[kind]) + rounding(ry), "dispatch backward")

    dr, dw = svt.svt_expert_combine_backward(dy, rows, pos, wd, out_rows=mark(T * K, D))
    rdr, rdw, mag = X.combine_backward(host(dy), hr, p, w, np.full((T * K, D), 7.0))
    near(host(dr), rdr, (U * (1 + 2 * HALF[kind]) + HALF[kind]) * np.abs(rdr) + TINY[kind], "d_rows")
    assert np.all(host(dr)[n:] == 7.0)
    near(host(dw), rdw, U * (D / 64 + 16) * mag + 2.0 ** -126, "d_weights")
    for a, b in zip((dr, dw), svt.svt_expert_combine_backward(dy, rows, pos, wd, out_rows=mark(T * K, D))):
        assert torch.equal(a, b)                  # the same bits again


def test_exchange_skips_foreign_positions(svt):
    x = dev(np.arange(6, dtype=np.float32).reshape(2, 3))
    pos = dev(np.array([[3, 4], [-1, 2 ** 31 - 1]], np.int32))
    out = svt.svt_expert_dispatch(x, pos, out=dev(np.full((4, 3), 7.0, np.float32)))
    assert host(out).tolist() == [[7, 7, 7], [7, 7, 7], [7, 7, 7], [0, 1, 2]]
    y = svt.svt_expert_combine(out, pos)
    assert host(y).tolist() == [[0, 1, 2], [0, 0, 0]]


def test_exchange_offsets_past_32_bits(svt):
    """Rows whose bytes and elements lie beyond 2^32: 2100 rows of 1 M float32 are 8.8 GB."""
    import torch
    T, K, D = 1050, 2, 1 << 20
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].expand(T, D).contiguous()
    pos = torch.arange(T * K, device="cuda", dtype=torch.int32).flip(0).view(T, K).contiguous()
    rows = svt.svt_expert_dispatch(x, pos)
    for t, j in ((0, 0), (0, 1), (T - 1, 0), (T - 1, 1), (500, 1)):
        assert bool((rows[int(pos[t, j])] == t).all())
    w = torch.full((T, K), 0.5, device="cuda")
    assert torch.equal(svt.svt_expert_combine(rows, pos, w), x)
    dr, dw = svt.svt_expert_combine_backward(x, rows, pos, w)
    assert bool((dr[int(pos[T - 1, 1])] == 0.5 * (T - 1)).all()) and bool((dr[int(pos[1, 0])] == 0.5).all())
    assert float(dw[1, 0]) == float(1 << 20) and float(dw[0, 0]) == 0.0


# ---- 4-bit products ----------------------------------------------------------------------------------

def make_weights(svt, rng, M, N, K, G, scale_kind, zeros, shift=0):
    groups = -(-K // G)
    nib = rng.integers(0, 256, (M, N, (K + 1) // 2)).astype(np.uint8)
    s = dev(rng.normal(size=(M, N, groups)) * 0.1, ty(scale_kind), shift)
    z = rng.integers(0, 16, (M, N, groups)).astype(np.uint8) if zeros else None
    packed = svt.svt_quant_pack(dev(nib, shift=3 * shift), s, None if z is None else dev(z, shift=shift), K, G)
    return packed, X.unpack(nib, K), host(s), z


LINEARS = [  # rows, outputs, inputs, group
    (1, 1, 1, 32), (1, 16, 128, 32), (2, 17, 33, 32), (16, 32, 256, 64), (17, 100, 127, 64), (13, 40, 129, 128),
    (5, 257, 1000, 128), (33, 64, 513, 32), (64, 48, 384, 64), (65, 130, 96, 32), (100, 33, 700, 128), (1, 512, 4097, 64),
    (150, 272, 320, 64), (300, 96, 1030, 32)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale_kind, zeros", [("f16", True), ("bf16", False), ("f32", True)])
@pytest.mark.parametrize("R, N, K, G", LINEARS)
def test_linear(svt, R, N, K, G, scale_kind, zeros, kind):
    say("linear", R, N, K, G, scale_kind, zeros, kind)
    rng = np.random.default_rng(R + N + K)
    shift = (R + N) % 2
    packed, q, s, z = make_weights(svt, rng, 1, N, K, G, scale_kind, zeros, shift)
    x = dev(rng.normal(size=(R, K)), ty(kind), shift)
    bias = rng.normal(size=(1, N)).astype(np.float32)
    parts = 3 if kind == "f32" else 1
    n = parts * G + -(-K // G) + 12
    for b, relu, out_kind in ((None, False, kind), (bias, True, kind), (bias, False, "f32")):
        y = svt.svt_quant_linear(x, packed, bias=None if b is None else dev(b), activation="relu" if relu else "none",
                                 out_dtype=ty(out_kind))
        ry, mag = X.linear(host(x), q, s, z, G, None, b, relu, np.zeros((R, N)))
        near(host(y), ry, 4 * np.sqrt(n) * U * mag + HALF[out_kind] * np.abs(ry) + TINY[out_kind], f"{relu} {out_kind}")


# sizes that reach every way the product is cut, each ending inside rows, outputs, blocks and groups
CUTS = [(1030, 4100, 260, 128), (520, 4000, 150, 64), (300, 3300, 137, 32), (13, 16400, 1100, 128), (5, 8200, 2050, 64), (16, 8200, 2050, 32), (16, 16400, 1100, 128), (16, 300, 4099, 64),
        (100, 2400, 259, 64), (9, 700, 1500, 128), (40, 600, 385, 32)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R, N, K, G", CUTS)
def test_linear_every_cut(svt, R, N, K, G, kind):
    say("cut", R, N, K, G, kind)
    rng = np.random.default_rng(R + N + K)
    packed, q, s, z = make_weights(svt, rng, 1, N, K, G, "bf16" if kind == "bf16" else "f32", R % 2 == 0)
    x = dev(rng.normal(size=(R, K)), ty(kind))
    bias = rng.normal(size=(1, N)).astype(np.float32)
    y = svt.svt_quant_linear(x, packed, bias=dev(bias), activation="relu")
    ry, mag = X.linear(host(x), q, s, z, G, None, bias, True, np.zeros((R, N)))
    n = (3 if kind == "f32" else 1) * G + -(-K // G) + 12
    near(host(y), ry, 4 * np.sqrt(n) * U * mag + HALF[kind] * np.abs(ry) + TINY[kind], "cut")


# sizes between the cuts' bounds: rows, outputs, inputs
BETWEEN = [(1031, 4100, 261), (1030, 4100, 7), (600, 4100, 33), (40, 11000, 261), (40, 2100, 1030), (40, 2100, 2101),
           (9, 700, 2101), (9, 5000, 1501), (3, 300, 1100)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("R, N, K", BETWEEN)
def test_linear_between_cuts(svt, R, N, K, G, kind):
    say("between", R, N, K, G, kind)
    rng = np.random.default_rng(R + N + K + G)
    packed, q, s, z = make_weights(svt, rng, 1, N, K, G, "f16" if kind == "f16" else "f32", (R + G // 32) % 2 == 0)
    x = dev(rng.normal(size=(R, K)) + 0.5, ty(kind))
    y = svt.svt_quant_linear(x, packed)
    ry, mag = X.linear(host(x), q, s, z, G, None, None, False, np.zeros((R, N)))
    n = (3 if kind == "f32" else 1) * G + -(-K // G) + 12
    near(host(y), ry, 4 * np.sqrt(n) * U * mag + HALF[kind] * np.abs(ry) + TINY[kind], "between")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("counts, N, K", [([200, 90, 33, 0, 250, 1, 140, 61], 4100, 261), ([90, 33, 0, 250], 4100, 130),
                                          ([3] * 30 + [0, 50], 1500, 389), ([1, 0, 2, 5], 40, 1030)])
def test_linear_by_expert_between_cuts(svt, counts, N, K, G, kind):
    say("experts between", counts[:5], N, K, G, kind)
    rng = np.random.default_rng(len(counts) + N + G)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1]) + 2
    packed, q, s, z = make_weights(svt, rng, len(counts), N, K, G, "f32", len(counts) % 8 == 0)
    xd = dev(rng.normal(size=(R, K)), ty(kind))
    y = svt.svt_quant_linear(xd, packed, offsets=dev(off), out=dev(np.full((R, N), 7.0), ty(kind)))
    ry, mag = X.linear(host(xd), q, s, z, G, off, None, False, np.full((R, N), 7.0))
    n = (3 if kind == "f32" else 1) * G + -(-K // G) + 12
    near(host(y), ry, 4 * np.sqrt(n) * U * mag + HALF[kind] * np.abs(ry) + TINY[kind], "experts between")
    assert np.all(host(y)[off[-1]:] == 7.0)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_linear_weights_are_exact(svt, kind, G):
    """Rows of the identity return the weights themselves: s (q - z), rounded once."""
    rng = np.random.default_rng(G)
    K, N = 150, 70
    packed, q, s, z = make_weights(svt, rng, 1, N, K, G, "f32", True)
    y = svt.svt_quant_linear(dev(np.eye(K), ty(kind)), packed, out_dtype=ty("f32"))
    sk, zk = np.repeat(s[0], G, 1)[:, :K], np.repeat(z[0].astype(np.float32), G, 1)[:, :K]
    want = (sk.astype(np.float32) * (q[0].astype(np.float32) - zk)).T
    assert np.array_equal(host(y).astype(np.float32), want)


EXPERTS = [  # rows per matrix, outputs, inputs, group
    ([1], 16, 64, 32), ([0, 3, 0, 1], 40, 130, 64), ([0, 0, 0], 16, 32, 32), ([17, 0, 40, 1, 16], 33, 256, 128),
    ([1] * 70, 16, 96, 32), ([0] * 63 + [5] + [0] * 100 + [2], 32, 64, 64), ([200, 7, 64], 100, 160, 32),
    ([130, 0, 65, 300], 200, 257, 64), ([40, 3], 50, 300, 128), ([0, 33], 16, 7, 32),
    ([1, 0, 2, 17] * 16, 2050, 300, 64), ([3] * 30 + [0, 50], 1500, 1030, 128), ([90, 33, 0, 250], 1030, 260, 128)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("counts, N, K, G", EXPERTS)
def test_linear_by_expert(svt, counts, N, K, G, kind):
    say("experts", counts[:5], N, K, G, kind)
    rng = np.random.default_rng(len(counts) + N)
    M, tail = len(counts), 3
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1]) + tail
    packed, q, s, z = make_weights(svt, rng, M, N, K, G, "bf16", True)
    x = rng.normal(size=(R, K))
    x[off[-1]:] = np.nan                          # rows behind the last one are not read
    xd, b = dev(x, ty(kind)), rng.normal(size=(M, N)).astype(np.float32)
    n = (3 if kind == "f32" else 1) * G + -(-K // G) + 12
    y = svt.svt_quant_linear(xd, packed, offsets=dev(off), bias=dev(b), activation="relu",
                             out=dev(np.full((R, N), 7.0), ty(kind)))
    ry, mag = X.linear(host(xd), q, s, z, G, off, b, True, np.full((R, N), 7.0))
    near(host(y), ry, 4 * np.sqrt(n) * U * mag + HALF[kind] * np.abs(ry) + TINY[kind], "experts")
    assert np.all(host(y)[off[-1]:] == 7.0)


@pytest.mark.parametrize("kind, unit", [("f16", 2.0 ** -24), ("bf16", 2.0 ** -120), ("f32", 2.0 ** -105)])
def test_linear_small_values_are_exact(svt, kind, unit):
    """Rows of the identity times a small unit (float16: its smallest subnormal; float32: with 24 significant
    bits): scales of 1, so every output is the unit times q - z, exactly."""
    K, N = 40, 48
    q = np.random.default_rng(3).integers(0, 16, (1, N, K)).astype(np.uint8)
    nib = dev((q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8))
    packed = svt.svt_quant_pack(nib, dev(np.ones((1, N, 2), np.float32)), None, K, 32)
    value = unit * ((2 ** 24 - 1) / 2 ** 23 if kind == "f32" else 1.0)
    y = svt.svt_quant_linear(dev(np.eye(K) * value, ty(kind)), packed, out_dtype=ty("f32"))
    if kind == "f32":   # 24 bits times 4 bits: rounded once more, and the start value 8 x once
        near(host(y), value * (q[0].astype(np.float64) - 8).T, 3 * U * 16 * value, "small")
    else:
        assert np.array_equal(host(y), value * (q[0].astype(np.float64) - 8).T)


def test_nothing_to_do(svt):
    """No tokens: empty outputs, offsets of 0; no rows: an empty product."""
    import torch
    e = torch.empty(0, 8, device="cuda", dtype=torch.float16)
    ids, w = svt.svt_route(e, 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert svt.svt_route_backward(e, ids, w, w).shape == (0, 8)
    off, order, pos = svt.svt_expert_sort(ids, 5)
    assert host(off).tolist() == [0] * 6 and order.shape == (0,) and pos.shape == (0, 2)
    rows = svt.svt_expert_dispatch(e, pos)
    assert rows.shape == (0, 8) and svt.svt_expert_combine(rows, pos, w).shape == (0, 8)
    assert svt.svt_expert_dispatch_backward(rows, pos).shape == (0, 8)
    assert [t.shape for t in svt.svt_expert_combine_backward(e, rows, pos, w)] == [(0, 8), (0, 2)]
    packed, *_ = make_weights(svt, np.random.default_rng(0), 5, 16, 8, 32, "f16", False)
    assert svt.svt_quant_linear(rows, packed, offsets=off).shape == (0, 16)


def test_refusals_leave_outputs(svt):
    """Calls that are refused on the device tensors themselves: errors, and outputs as they were."""
    import torch
    f = torch.ones(4, 8, device="cuda")
    i = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    rows, w = torch.ones(8, 8, device="cuda"), torch.ones(4, 2, device="cuda")
    out = torch.full((8, 8), 7.0, device="cuda")
    packed, *_ = make_weights(svt, np.random.default_rng(0), 2, 16, 8, 32, "f16", False)
    for call in [
        lambda: svt.svt_route(f, 9), lambda: svt.svt_route(f, 0), lambda: svt.svt_route(f, -1),
        lambda: svt.svt_route_backward(f, i[:3], w, w), lambda: svt.svt_route_backward(f, i, w.half(), w),
        lambda: svt.svt_expert_sort(i, 0), lambda: svt.svt_expert_sort(i, 513), lambda: svt.svt_expert_sort(i, -4),
        lambda: svt.svt_expert_dispatch(f, i[:2], out=out), lambda: svt.svt_expert_dispatch(f, i, out=out[:4]),
        lambda: svt.svt_expert_dispatch(out[:4], i, out=out),
        lambda: svt.svt_expert_combine(rows[:6], i, w), lambda: svt.svt_expert_combine(out, i, w, out=out[:4]),
        lambda: svt.svt_expert_combine_backward(f, rows.half(), i, w, out_rows=out),
        lambda: svt.svt_expert_combine_backward(f, rows, i, w, out_rows=rows),
        lambda: svt.svt_quant_linear(f, packed, out=out), lambda: svt.svt_quant_linear(f[:, :4], packed),
        lambda: svt.svt_quant_linear(f, packed, offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: svt.svt_quant_linear(f, packed, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"),
                                     activation="gelu"),
        lambda: svt.svt_quant_linear(f, packed, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"),
                                     out_dtype=torch.float16),
        lambda: svt.svt_quant_pack(torch.zeros(16, 3, dtype=torch.uint8, device="cuda"), rows[:, :1], None, 8, 32),
        lambda: svt.svt_quant_pack(torch.zeros(8, 4, dtype=torch.uint8, device="cuda"), rows[:, :1].contiguous(), None, 8, 16),
    ]:
        with pytest.raises((ValueError, svt.SvtError)):
            call()
    torch.cuda.synchronize()
    assert bool((out == 7.0).all()) and bool((rows == 1.0).all())


def test_linear_more_units_than_one_grid(svt):
    """1,100,000 rows by 3 experts: more blocks of rows than one grid dimension takes; rows around its end and
    the experts' are compared."""
    import torch
    R, N, K = 1100000, 16, 32
    rng = np.random.default_rng(2)
    packed, q, s, z = make_weights(svt, rng, 3, N, K, 32, "f16", True)
    x = torch.randn(R, K, device="cuda").half()
    off = np.array([0, 5, 1048570, R], np.int32)
    y = svt.svt_quant_linear(x, packed, offsets=dev(off))
    pick = np.array([0, 4, 5, 6, 1000, 524287, 524288, 1048560, 1048569, 1048570, 1048580, 1048608, R - 1])
    hx, hy = host(x[pick]), host(y[pick])
    for i, r in enumerate(pick):
        e = int(np.searchsorted(off, r, side="right")) - 1
        ry, mag = X.linear(hx[i:i + 1], q[e:e + 1], s[e:e + 1], z[e:e + 1], 32, None, None, False, np.zeros((1, N)))
        near(hy[i:i + 1], ry, 4 * np.sqrt(45) * U * mag + HALF["f16"] * np.abs(ry) + TINY["f16"], f"row {r}")


def test_linear_offsets_are_clamped(svt):
    """Ends past the rows are cut, ends that do not ascend give no rows; nothing else is touched."""
    rng = np.random.default_rng(8)
    packed, q, s, z = make_weights(svt, rng, 3, 16, 32, 32, "f32", False)
    x = rng.normal(size=(6, 32)).astype(np.float32)
    for off in ([-5, 2, 2 ** 31 - 1, 7], [4, 1, 3, 3], [2 ** 31 - 1] * 4, [-2 ** 31] * 4):
        off = np.array(off, np.int32)
        y = svt.svt_quant_linear(dev(x), packed, offsets=dev(off), out=dev(np.full((6, 16), 7.0, np.float32)))
        ry, mag = X.linear(x, q, s, z, 32, off, None, False, np.full((6, 16), 7.0))
        near(host(y), ry, 4 * np.sqrt(110) * U * mag + U * np.abs(ry), f"offsets {off}")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_linear_infinity_and_nan_stay_in_their_row(svt, kind):
    rng = np.random.default_rng(9)
    packed, q, s, z = make_weights(svt, rng, 1, 40, 200, 64, "f16", True)
    x = rng.normal(size=(5, 200))
    x[1, 7], x[3, 199] = np.inf, np.nan
    for act in ("none", "relu"):
        y = host(svt.svt_quant_linear(dev(x, ty(kind)), packed, activation=act))
        assert np.all(np.isnan(y[[1, 3]])) and np.all(np.isfinite(y[[0, 2, 4]]))


# ---- together ----------------------------------------------------------------------------------------

def net(rng, svt, E, D, H, G):
    up = make_weights(svt, rng, E, H, D, G, "f16", True)
    down = make_weights(svt, rng, E, D, H, G, "f16", False)
    bias = rng.normal(size=(E, H)).astype(np.float32)
    return up, down, bias


def routed(svt, x, logits, K, up, down, bias, s=None):
    """One layer of routed experts as a serving program runs it."""
    E = logits.shape[1]
    ids, w = svt.svt_route(logits, K, stream=s)
    off, order, pos = svt.svt_expert_sort(ids, E, stream=s)
    rows = svt.svt_expert_dispatch(x, pos, stream=s)
    h = svt.svt_quant_linear(rows, up, offsets=off, bias=bias, activation="relu", stream=s)
    o = svt.svt_quant_linear(h, down, offsets=off, stream=s)
    return svt.svt_expert_combine(o, pos, w, stream=s)


def routed_oracle(x, logits, K, G, up, down, bias):
    T, E = logits.shape
    ids, w, _ = X.route(logits, K, True)
    off, _, pos = X.sort(ids, E)
    rows = X.dispatch(x, pos, np.zeros((T * K, x.shape[1])))
    h, hm = X.linear(rows, up[1], up[2], up[3], G, off, bias, True, np.zeros((T * K, bias.shape[1])))
    o, om = X.linear(h, down[1], down[2], down[3], G, off, None, False, np.zeros((T * K, x.shape[1])))
    _, spread = X.linear(hm, down[1], np.abs(down[2]), None, G, off, None, False, np.zeros((T * K, x.shape[1])))
    y, _ = X.combine(o, pos, w)
    _, mag = X.combine(om + spread, pos, w)
    return y, mag


@pytest.mark.parametrize("T", [1, 50, 700])
def test_routed_layer(svt, T):
    """Route, sort, dispatch, two products and combine in float32.  Errors of the first product (4 sqrt(n) u of
    its magnitudes) pass the second as magnitudes do; the weights add their own relative 60 u."""
    rng = np.random.default_rng(T)
    E, D, H, K, G = 6, 64, 96, 2, 32
    up, down, bias = net(rng, svt, E, D, H, G)
    x, logits = rng.normal(size=(T, D)).astype(np.float32), rng.normal(size=(T, E)).astype(np.float32)
    y = routed(svt, dev(x), dev(logits), K, up[0], down[0], dev(bias))
    ry, mag = routed_oracle(x.astype(np.float64), logits, K, G, up, down, bias)
    n = 3 * G + 3 + 12
    near(host(y), ry, (4 * np.sqrt(n) + 60) * U * mag, "layer")


def test_rerank_candidates_through_a_routed_net(svt):
    """The candidates of a search, each sent to 2 of 6 experts by its own interaction with the query."""
    import oracle_pins as P
    rng = np.random.default_rng(4)
    items, sigs, cl, cent = P.small_catalogue(rng, n=3000, d=64, nlist=8, W=2)
    ix = svt.Index(items, sigs, cl, cent, 1.0)
    q = rng.integers(-127, 128, (2, 64)).astype(np.int8)
    m = np.zeros((2, 2), np.int64)
    ids, *_ = ix.search(dev(q), dev(m), 4, 100)
    c = host(ids)
    assert np.all(c >= 0)
    z = (items[c].astype(np.float32) * q[:, None, :].astype(np.float32) / 127.0 ** 2).reshape(200, 64)
    E, H, K, G = 6, 48, 2, 32
    up, down, bias = net(rng, svt, E, 64, H, G)
    gate = rng.normal(size=(64, E)).astype(np.float32)
    logits = z @ gate
    y = routed(svt, dev(z), dev(logits), K, up[0], down[0], dev(bias))
    ry, mag = routed_oracle(z.astype(np.float64), logits, K, G, up, down, bias)
    near(host(y), ry, (4 * np.sqrt(3 * G + 14) + 60) * U * mag, "scores")
    ix.close()


def test_training_step_gradients_against_differences(svt):
    """The gradients of sum(dy * y) through combine, one expert scale per expert, dispatch and the router, in
    the order a training step runs them, against differences of the float64 oracle."""
    rng = np.random.default_rng(12)
    T, E, K, D = 12, 5, 2, 16
    x, logits = rng.normal(size=(T, D)).astype(np.float32), (2 * rng.normal(size=(T, E))).astype(np.float32)
    dy, gain = rng.normal(size=(T, D)).astype(np.float32), rng.normal(size=(E, D)).astype(np.float32)

    def loss(x, logits):
        ids, w, _ = X.route(logits, K, True)
        _, _, pos = X.sort(ids, E)
        rows = X.dispatch(x, pos, np.zeros((T * K, D)))
        owner = np.zeros(T * K, int)
        owner[pos.reshape(-1)] = ids.reshape(-1)
        y, _ = X.combine(rows * gain[owner], pos, w)
        return float(np.sum(y * dy)), ids

    xd, ld = dev(x), dev(logits)
    ids, w = svt.svt_route(ld, K)
    off, order, pos = svt.svt_expert_sort(ids, E)
    rows = svt.svt_expert_dispatch(xd, pos)
    owner = ids.reshape(-1)[order.long()].long()
    scaled = rows * dev(gain)[owner]
    d_scaled, dw = svt.svt_expert_combine_backward(dev(dy), scaled, pos, w)
    dx = svt.svt_expert_dispatch_backward(d_scaled * dev(gain)[owner], pos)
    dl = svt.svt_route_backward(ld, ids, w, dw)
    x64, l64, h = x.astype(np.float64), logits.astype(np.float64), 1e-5
    _, base = loss(x64, l64)
    for arr, got in ((x64, host(dx)), (l64, host(dl))):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            f = []
            for step in (h, -h):
                arr[i] = keep + step
                v, ids2 = loss(x64, l64)
                assert np.array_equal(ids2, base)
                f.append(v)
            arr[i] = keep
            # float32 gradients of sums of about 16 terms of size 1..10, differences good to h^2
            assert abs((f[0] - f[1]) / (2 * h) - got[i]) < 2e-5


def test_captured_layer_replays(svt):
    """The layer captured into a graph: every replay, on new inputs in place and with eager work between, equals
    the eager result bit for bit; two graphs keep their workspaces apart."""
    import torch
    rng = np.random.default_rng(6)
    E, D, H, K, G, T = 40, 64, 64, 2, 64, 10000   # 20000 entries: the sort with a workspace
    up, down, bias = net(rng, svt, E, D, H, G)
    b = dev(bias)
    graphs = []
    for i in range(2):
        x, l = torch.zeros(T, D, device="cuda", dtype=torch.bfloat16), torch.zeros(T, E, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            routed(svt, x, l, K, up[0], down[0], b)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = routed(svt, x, l, K, up[0], down[0], b)
        graphs.append((g, x, l, y))
    for step in range(4):
        wants = []
        for g, x, l, y in graphs:
            x.copy_(torch.randn(T, D, device="cuda"))
            l.copy_(torch.randn(T, E, device="cuda"))
            wants.append(routed(svt, x, l, K, up[0], down[0], b))
        torch.cuda.synchronize()
        for g, *_ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (g, x, l, y), want in zip(graphs, wants):
            assert torch.equal(y, want), f"replay {step}"


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_captured_gradients_and_products_replay(svt, kind):
    """Every gradient call and a large product captured into one graph: each replay, on inputs changed in place
    and with the same calls run eagerly between, gives the eager bits."""
    import torch
    T, E, K, D, N = 1100, 20, 3, 200, 2100
    rng = np.random.default_rng(13)
    packed, *_ = make_weights(svt, rng, 1, N, D, 32, "f32", True)
    logits, dy = torch.zeros(T, E, device="cuda", dtype=ty(kind)), torch.zeros(T, D, device="cuda", dtype=ty(kind))
    rows = torch.zeros(T * K, D, device="cuda", dtype=ty(kind))

    def step():
        ids, w = svt.svt_route(logits, K, renormalise=False)
        off, order, pos = svt.svt_expert_sort(ids, E)
        dr, dw = svt.svt_expert_combine_backward(dy, rows, pos, w)
        dx = svt.svt_expert_dispatch_backward(dr, pos)
        dl = svt.svt_route_backward(logits, ids, w, dw, renormalise=False)
        return ids, w, off, order, pos, dr, dw, dx, dl, svt.svt_quant_linear(dy, packed)

    def change():
        for t in (logits, dy, rows):
            t.copy_(torch.randn(t.shape, device="cuda"))

    change()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(4):
        change()
        want = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {i}"


def test_layer_on_another_stream(svt):
    import torch
    rng = np.random.default_rng(7)
    E, D, H, K, G, T = 12, 64, 64, 3, 32, 9000
    up, down, bias = net(rng, svt, E, D, H, G)
    x, l, b = dev(rng.normal(size=(T, D)), ty("f16")), dev(rng.normal(size=(T, E)), ty("f16")), dev(bias)
    want = routed(svt, x, l, K, up[0], down[0], b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [routed(svt, x, l, K, up[0], down[0], b, s) for _ in range(3) for s in streams]   # both at once
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
