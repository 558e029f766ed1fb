"""Gated products and embedding gradients of small whole numbers on the GPU: every product and every float32 sum is exact, whatever its order, so
that the results are the float64 definition's, rounded once.  A part that is lost or counted twice shows."""
import numpy as np
import pytest

from gpu_common import say
from test_gpu_scorer_gated import offsets_for, svt, ty   # noqa: F401 (svt is a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture
def give_back():
    """The memory of a large case, to those that do not allocate through torch."""
    yield
    import torch
    torch.cuda.empty_cache()


def whole(g, kind, *shape):
    import torch
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8).to(ty(kind))


def compare(svt, R, K, N, M, act, kind, how):   # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(R + 3 * K + 5 * N + 7 * M)
    o = [0, R] if M == 0 else offsets_for(np.random.default_rng(R + M), R, M, how).tolist()
    od = torch.tensor(o, dtype=torch.int32, device="cuda") if M else None
    shape = (M, N, K) if M else (N, K)
    x, dh, gate, up = (whole(g, kind, R, n) for n in (K, N, N, N))
    wg, wu = whole(g, kind, *shape), whole(g, kind, *shape)
    h, a, b = svt.svt_gated_linear(x, wg, wu, offsets=od, activation=act, keep=True)
    dx, dwg, dwu = svt.svt_gated_linear_backward(dh, x, wg, wu, gate, up, offsets=od, activation=act)
    dwg, dwu, wg, wu = (t.view(max(M, 1), N, K) for t in (dwg, dwu, wg, wu))
    for e in range(max(M, 1)):
        r = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            assert not dwg[e].any() and not dwu[e].any(), e
            continue
        X, G, W = x[r].double(), gate[r].double(), [t[e].double() for t in (wg, wu)]
        pa, pb = X @ W[0].T, X @ W[1].T
        assert torch.equal(a[r], pa.to(ty(kind))) and torch.equal(b[r], pb.to(ty(kind))), e
        product = (pa.clamp(min=0) if act == "relu" else pa).float() * pb.float()   # the one float32 rounding
        assert torch.equal(h[r], product.to(ty(kind))), e
        dg = dh[r].double() * up[r].double() * ((G > 0) if act == "relu" else 1)
        du = dh[r].double() * (G.clamp(min=0) if act == "relu" else G)
        assert torch.equal(dx[r], (dg @ W[0] + du @ W[1]).to(ty(kind))), e
        assert torch.equal(dwg[e], (dg.T @ X).to(ty(kind))) and torch.equal(dwu[e], (du.T @ X).to(ty(kind))), e


# dense and by expert: one tile, several, sums in parts, long experts, tiles of every cut
SIZES = [(1, 70, 40, 0, ""), (64, 300, 200, 0, ""), (1001, 250, 999, 0, ""), (300, 2000, 33, 0, ""), (4100, 72, 1544, 0, ""),
         (40, 64, 64, 9, "uneven"), (2048, 128, 256, 8, "uneven"), (9000, 40, 24, 70, "uneven"), (20000, 24, 20, 3, "one"),
         (16384, 256, 512, 8, "uneven"), (700, 36, 20, 512, "even")]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_whole_numbers(svt, size, kind):   # noqa: F811
    say("whole numbers", size, kind)
    compare(svt, *size[:4], "none" if size[0] % 2 else "relu", kind, size[4])


# more workgroups than a grid has along one side: gradients of many experts with long outputs
@pytest.mark.parametrize("R, K, N, M", [(64, 16, 1 << 20, 64), (1000, 64, 131072, 512)])
def test_more_workgroups_than_a_grid_row(svt, give_back, R, K, N, M):   # noqa: F811
    say("grid rows", R, K, N, M)
    compare(svt, R, K, N, M, "none", "bf16", "uneven")


@pytest.mark.parametrize("M", [0, 3])
def test_the_most_rows(svt, give_back, M):   # noqa: F811
    """2^31 - 1 rows of one value: rows far past what one side of a grid numbers.  The sums over rows stay below 2^24: they
    are random walks of 2^31 steps of about 8."""
    import torch
    say("most rows", M)
    R = 2 ** 31 - 1
    g = torch.Generator(device="cuda").manual_seed(7)
    o = [5, R // 3, R // 3, R - 9] if M else [0, R]
    od = torch.tensor(o, dtype=torch.int32, device="cuda") if M else None
    x, dh, gate, up = (whole(g, "f32", R, 1) for _ in range(4))
    wg = torch.tensor([2.0, 3.0, -1.0][:max(M, 1)], device="cuda").view(*(M, 1, 1) if M else (1, 1))
    wu = torch.tensor([-1.0, 2.0, 3.0][:max(M, 1)], device="cuda").view_as(wg)
    h = svt.svt_gated_linear(x, wg, wu, offsets=od, activation="none")
    for e in range(max(M, 1)):
        r = slice(o[e], o[e + 1])
        assert torch.equal(h[r], x[r] * x[r] * (wg.view(-1)[e] * wu.view(-1)[e])), e
    del h
    dx, dwg, dwu = svt.svt_gated_linear_backward(dh, x, wg, wu, gate, up, offsets=od, activation="none")
    for e in range(max(M, 1)):
        r = slice(o[e], o[e + 1])
        assert torch.equal(dx[r], dh[r] * (up[r] * wg.view(-1)[e] + gate[r] * wu.view(-1)[e])), e
        for dw, other in ((dwg, up), (dwu, gate)):
            want = sum((dh[a:b] * other[a:b] * x[a:b]).sum(dtype=torch.float64)
                       for a in range(o[e], o[e + 1], 1 << 27) for b in (min(a + (1 << 27), o[e + 1]),))
            assert dw.view(-1)[e].item() == float(want), e


def test_embedding_gradient_of_more_workgroups_than_a_grid_row(svt, give_back):   # noqa: F811
    """Rows of 2^24 - 1 float16, which begin at 2 bytes: 138 chunks of 8 places and 2^17 pieces of a row's columns each, four to
    a workgroup."""
    import torch
    n, V, D = 1101, 4, 2 ** 24 - 1
    say("wide rows", n, V, D)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(-1, V, (n,), generator=g, device="cuda")
    ids[ids == 2] = 3   # a row that no token names, and runs over many chunks
    d = whole(g, "f16", n, D)
    out = svt.svt_embedding_backward(d, ids, V)
    given = whole(g, "f16", V, D)
    added = svt.svt_embedding_backward(d, ids, V, out=given.clone(), accumulate=True)
    for v in range(V):
        want = torch.zeros(D, device="cuda")
        for i in (ids == v).nonzero()[:, 0].tolist():
            want += d[i]
        assert torch.equal(out[v], want.half()), v
        assert torch.equal(added[v], (want + given[v]).half()), v
