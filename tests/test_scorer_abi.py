"""Entry points of the trained scorer's operators: every documented refusal, on the host (nothing is enqueued: the
pointers are never read), workspace sizes, and the binding's checks of tensors."""
import pytest

from int8_ivf_ann_amd import svt

P = [0x100000000 * (i + 1) for i in range(12)]   # disjoint, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(svt.LIB_PATH):
        from int8_ivf_ann_amd import build
        build.build()
    return svt.lib()


def refused(rc, code=svt.SVT_EINVAL, text=None):
    assert rc == code, (rc, svt.svt_last_error())
    msg = svt.svt_last_error()
    assert msg and (text is None or text in msg), msg


SIZES = [(dict(T=-1), "n_tokens"), (dict(T=2 ** 30 + 1), "n_tokens"), (dict(V=0), "n_rows"), (dict(V=2 ** 31 - 1), "n_rows"),
         (dict(D=0), "width"), (dict(D=2 ** 24 + 1), "width"), (dict(dtype=3), "type"), (dict(scale=float("nan")), "finite"),
         (dict(scale=float("inf")), "finite")]


@pytest.mark.parametrize("kw, text", SIZES + [
    *[(dict([(i, None)]), "NULL") for i in range(3)], *[(dict([(i, P[i] + 1)]), "misaligned") for i in range(3)],
    (dict([(2, P[0] + 64)]), "overlap"), (dict([(2, P[1])]), "overlap")])
def test_embedding_refusals(L, kw, text):
    v = dict(T=64, V=100, D=24, dtype=svt.SVT_F16, scale=1.0)
    v.update({i: P[i] for i in range(3)})
    v.update(kw)
    refused(L.svt_embedding(v["T"], v["V"], v["D"], v["dtype"], v[0], v[1], v["scale"], v[2], None), text=text)


@pytest.mark.parametrize("kw, text", SIZES + [
    *[(dict([(i, None)]), "NULL") for i in range(3)], *[(dict([(i, P[i] + 1)]), "misaligned") for i in range(3)],
    (dict(ws=P[3] + 8), "misaligned"), (dict(acc=2), "accumulate"), (dict(acc=-1), "accumulate"), (dict(td=svt.SVT_BF16), "type"),
    (dict(td=9), "type"), (dict(ws=None), "workspace"), (dict(nb=16), "workspace"), (dict([(2, P[0] + 64)]), "overlap"),
    (dict([(2, P[1])]), "overlap"), (dict(ws=P[2]), "overlap"), (dict(ws=P[0] + 16), "overlap")])
def test_embedding_backward_refusals(L, kw, text):
    v = dict(T=64, V=100, D=24, dtype=svt.SVT_F16, scale=1.0, acc=0, td=svt.SVT_F32, ws=P[3], nb=1 << 24)
    v.update({i: P[i] for i in range(3)})
    v.update(kw)
    refused(L.svt_embedding_backward(v["T"], v["V"], v["D"], v["dtype"], v[0], v[1], v["scale"], v["acc"], v["td"], v[2], v["ws"],
                                     v["nb"], None), text=text)


def test_embedding_workspace_size(L):
    assert L.svt_embedding_backward_workspace_size(0, 10, 8) == 0 and not svt.svt_last_error()
    for n, V, D in ((1, 1, 1), (8192, 1000, 64), (8193, 1 << 20, 64), (1 << 20, 5, 128), (1 << 22, 2 ** 31 - 2, 16)):
        need = L.svt_embedding_backward_workspace_size(n, V, D)
        # keys and order twice, partial sums of at most one chunk of 8 tokens, histograms
        assert 8 * n < need <= 16 * n + (n // 8 + 1) * (8 * D + 4) + (1 << 20), (n, V, D, need)
        assert svt.svt_embedding_backward_workspace_size(n, V, D) == need
    assert svt.svt_embedding_backward_workspace_size(1 << 30, 1 << 30, 64) > 1 << 33
    for bad in ((-1, 10, 8), (1, 0, 8), (1, 10, 0)):
        assert L.svt_embedding_backward_workspace_size(*bad) == 0 and svt.svt_last_error()
        with pytest.raises(svt.SvtError):
            svt.svt_embedding_backward_workspace_size(*bad)


ROWS = [(dict(T=-1), "n_tokens"), (dict(V=0), "vocab"), (dict(V=2 ** 30 + 1), "vocab"), (dict(dtype=7), "type"),
        (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"),
        (dict(scale=float("inf")), "scale")]


@pytest.mark.parametrize("kw, text", ROWS + [
    (dict(top=-1), "top"), (dict(top=17), "top"), (dict(V=3, top=4), "top"), *[(dict([(i, None)]), "NULL") for i in range(7)],
    (dict([(0, P[0] + 1)]), "misaligned"), (dict([(1, P[1] + 4)]), "misaligned"), (dict([(3, P[3] + 2)]), "misaligned"),
    (dict([(5, P[5] + 4)]), "misaligned"), (dict(ws=P[7] + 4), "misaligned"), (dict([(2, P[0] + 8)]), "overlap"),
    (dict([(4, P[3])]), "overlap"), (dict([(6, P[1])]), "overlap"), (dict(V=100000, ws=None), "workspace"),
    (dict(V=100000, nb=64), "workspace"), (dict(V=100000, ws=P[5]), "overlap")])
def test_logprobs_refusals(L, kw, text):
    v = dict(T=4, V=64, top=2, dtype=svt.SVT_F16, scale=1.0, ws=P[7], nb=1 << 20)
    v.update({i: P[i] for i in range(7)})
    v.update(kw)
    refused(L.svt_token_logprobs(v["T"], v["V"], v["top"], v["dtype"], v[0], v[1], v["scale"], v[2], v[3], v[4], v[5], v[6],
                                 v["ws"], v["nb"], None), text=text)


@pytest.mark.parametrize("kw, text", ROWS + [
    *[(dict([(i, None)]), "NULL") for i in (0, 1, 2, 3, 4, 6)], *[(dict([(i, P[i] + 1)]), "misaligned") for i in range(7)],
    *[(dict([(6, P[i])]), "overlap") for i in range(6)]])
def test_logprobs_backward_refusals(L, kw, text):
    v = dict(T=4, V=64, dtype=svt.SVT_BF16, scale=1.0)
    v.update({i: P[i] for i in range(7)})
    v.update(kw)
    refused(L.svt_token_logprobs_backward(v["T"], v["V"], v["dtype"], v[0], v[1], v["scale"], v[2], v[3], v[4], v[5], v[6], None),
            text=text)


def test_logprobs_workspace_size(L):
    assert L.svt_token_logprobs_workspace_size(1000, 50000, 8) == 0 and not svt.svt_last_error()
    assert 0 < L.svt_token_logprobs_workspace_size(1, 131072, 16) < 1 << 20
    assert L.svt_token_logprobs_workspace_size(0, 10, 0) == 0 and not svt.svt_last_error()
    for bad in ((-1, 10, 0), (1, 0, 0), (1, 10, 11), (1, 100, 17)):
        assert L.svt_token_logprobs_workspace_size(*bad) == 0 and svt.svt_last_error()
        with pytest.raises(svt.SvtError):
            svt.svt_token_logprobs_workspace_size(*bad)


GATED = [(dict(R=-1), "n_rows"), (dict(K=0), "n_in"), (dict(K=2 ** 20 + 1), "n_in"), (dict(N=0), "n_out"),
         (dict(N=2 ** 20 + 1), "n_out"), (dict(M=0), "n_matrices"), (dict(M=513), "n_matrices"), (dict(dtype=3), "type"),
         (dict(act=4), "activation"), (dict(act=-1), "activation"), (dict(M=2, off=None), "offsets"),
         (dict(off=P[11] + 2), "misaligned")]


@pytest.mark.parametrize("kw, text", GATED + [
    *[(dict([(i, None)]), "NULL") for i in range(4)], (dict([(4, None)]), "both or neither"),
    (dict([(5, None)]), "both or neither"), *[(dict([(i, P[i] + 1)]), "misaligned") for i in range(6)],
    (dict(ws=P[9] + 4), "misaligned"), (dict([(3, P[0] + 8)]), "overlap"), (dict([(4, P[3])]), "overlap"),
    (dict([(5, P[1])]), "overlap"), (dict([(3, P[11])]), "overlap"),
    (dict(R=400, K=33, ws=None), "workspace"), (dict(R=400, K=33, nb=64), "workspace"), (dict(R=400, K=33, ws=P[3]), "overlap"),
    (dict(R=400, ws=None, x=2), "workspace"), (dict(R=2 ** 31 - 1, N=2 ** 20), "too many rows")])
def test_gated_refusals(L, kw, text):
    v = dict(R=64, K=32, N=16, M=2, dtype=svt.SVT_F16, act=svt.SVT_ACT_SILU, off=P[11], ws=P[9], nb=1 << 24, x=0)
    v.update({i: P[i] for i in range(6)})
    if kw.get("R") == 2 ** 31 - 1:   # far apart, so that only the size is wrong
        v.update({i: (i + 1) << 52 for i in range(6)})
    v.update(kw)
    refused(L.svt_gated_linear(v["R"], v["K"], v["N"], v["M"], v["dtype"], v[0] + v["x"] if v[0] else None, v[1], v[2], v["off"],
                               v["act"], v[3], v[4], v[5], v["ws"], v["nb"], None), text=text)


@pytest.mark.parametrize("kw, text", GATED + [
    *[(dict([(i, None)]), "NULL") for i in range(6)], (dict([(7, None)]), "both or neither"), (dict([(8, None)]), "both or neither"),
    (dict([(6, None), (7, None), (8, None)]), "NULL"), *[(dict([(i, P[i] + 1)]), "misaligned") for i in range(9)],
    (dict(ws=P[9] + 8), "misaligned"), (dict(ws=None), "workspace"), (dict(nb=256), "workspace"),
    *[(dict([(6, P[i])]), "overlap") for i in range(6)], (dict([(7, P[6])]), "overlap"), (dict([(8, P[7])]), "overlap"),
    (dict([(8, P[11])]), "overlap"), (dict(ws=P[0]), "overlap"), (dict(ws=P[8]), "overlap")])
def test_gated_backward_refusals(L, kw, text):
    v = dict(R=64, K=32, N=16, M=2, dtype=svt.SVT_BF16, act=svt.SVT_ACT_GELU, off=P[11], ws=P[9], nb=1 << 24)
    v.update({i: P[i] for i in range(9)})
    v.update(kw)
    refused(L.svt_gated_linear_backward(v["R"], v["K"], v["N"], v["M"], v["dtype"], *[v[i] for i in range(6)], v["off"],
                                        v["act"], v[6], v[7], v[8], v["ws"], v["nb"], None), text=text)


def test_gated_workspace_size(L):
    size, grad = L.svt_gated_linear_workspace_size, L.svt_gated_linear_backward_workspace_size
    assert size(400, 32, 16, 1, svt.SVT_F16, 0, 1) == 0 and not svt.svt_last_error()
    assert size(400, 33, 16, 1, svt.SVT_F32, 0, 1) == 0                       # 4-byte rows as they are
    assert size(400, 33, 16, 1, svt.SVT_F16, 0, 1) == (400 + 32) * 80         # copies with rows of 80 bytes
    assert size(400, 32, 16, 1, svt.SVT_F16, 0, 0) == (400 + 32) * 64
    assert size(20, 33, 16, 1, svt.SVT_F16, 0, 1) == 0                        # few rows: never copied
    assert size(0, 33, 16, 1, svt.SVT_F16, 0, 0) == 0
    assert grad(0, 33, 16, 1, svt.SVT_F16, 0, 0) == 0 and not svt.svt_last_error()
    both = 2 * 400 * 32
    assert grad(400, 32, 16, 1, svt.SVT_F16, 0, 1) >= both
    assert grad(400, 32, 16, 1, svt.SVT_F16, 0, 0) - grad(400, 32, 16, 1, svt.SVT_F16, 0, 1) == (400 + 32) * 64
    for f in (size, grad):
        for bad in ((-1, 8, 8, 1, 0, 0, 1), (1, 0, 8, 1, 0, 0, 1), (1, 8, 8, 2, 0, 0, 1), (1, 8, 8, 513, 0, 1, 1),
                    (1, 8, 8, 1, 5, 0, 1)):
            assert f(*bad) == 0 and svt.svt_last_error()
    n = 2 ** 31 - 1   # dg and du with rows of 16 bytes, copies of x and both weights
    assert grad(n, 1, 1, 1, svt.SVT_F16, 0, 1) >= 2 * n * 16 + (n + 2) * 16
    assert svt.svt_gated_linear_workspace_size(n, 1, 1, 1, svt.SVT_F16, False, True) == (n + 2) * 16
    assert svt.svt_gated_linear_backward_workspace_size(n, 1, 1, 1, svt.SVT_F16, False, True) == grad(n, 1, 1, 1, svt.SVT_F16, 0, 1)
    with pytest.raises(svt.SvtError):
        svt.svt_gated_linear_workspace_size(1, 0, 8, 1, 0, False, True)
    with pytest.raises(svt.SvtError):
        svt.svt_gated_linear_backward_workspace_size(1, 0, 8, 1, 0, False, True)


# ---- the binding -------------------------------------------------------------------------------------

def test_tensors_that_require_grad_or_lie_on_the_host_are_refused():
    import torch
    f = torch.zeros((4, 8), requires_grad=True)
    i, v = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    w = torch.zeros((8, 8))
    calls = [lambda: svt.svt_embedding(f, i), lambda: svt.svt_embedding_backward(f, i, 5),
             lambda: svt.svt_gated_linear(f, w, w), lambda: svt.svt_gated_linear_backward(f, f, w, w, f, f),
             lambda: svt.svt_token_logprobs(f, i), lambda: svt.svt_token_logprobs_backward(f, i, f, v, v)]
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):   # the next check
            call()


class Stand:
    """A device tensor's attributes, without a device or storage."""
    is_cuda, requires_grad = True, False

    def __init__(self, dtype, *shape, contiguous=True):
        import torch
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda", 0)
        self.contiguous = contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 0x1000


def test_shapes_and_types_are_checked():
    import torch
    f32, bf16, i64, i32 = torch.float32, torch.bfloat16, torch.int64, torch.int32
    table, ids = Stand(bf16, 10, 8), Stand(i64, 4)
    bad = [
        (lambda: svt.svt_embedding(Stand(torch.float64, 10, 8), ids), "table"),
        (lambda: svt.svt_embedding(Stand(bf16, 10), ids), "table"),
        (lambda: svt.svt_embedding(Stand(bf16, 10, 8, contiguous=False), ids), "table"),
        (lambda: svt.svt_embedding(table, Stand(i32, 4)), "ids"),
        (lambda: svt.svt_embedding(table, Stand(i64, 4, 2, contiguous=False)), "ids"),
        (lambda: svt.svt_embedding(table, [1, 2]), "ids"),
        (lambda: svt.svt_embedding_backward(Stand(bf16, 4, 8), Stand(i64, 5), 10), "ids"),
        (lambda: svt.svt_embedding_backward(Stand(bf16, 4, 8), Stand(i64, 4), 10, accumulate=True), "out"),
        (lambda: svt.svt_embedding_backward(Stand(bf16, 4, 8), Stand(i64, 4), 10, out_dtype=torch.float16), "out"),
        (lambda: svt.svt_embedding_backward(Stand(bf16, 4, 8), Stand(i64, 4), 10, out=Stand(bf16, 10, 8), out_dtype=f32), "out"),
        (lambda: svt.svt_embedding_backward(3.0, Stand(i64, 4), 10), "d_out"),
        (lambda: svt.svt_token_logprobs(Stand(bf16, 4, 8), Stand(i32, 4)), "tokens"),
        (lambda: svt.svt_token_logprobs(Stand(bf16, 4, 8), Stand(i64, 5)), "tokens"),
        (lambda: svt.svt_token_logprobs(Stand(bf16, 4, 8), Stand(i64, 4), top=9), "top"),
        (lambda: svt.svt_token_logprobs(Stand(bf16, 4, 80), Stand(i64, 4), top=17), "top"),
        (lambda: svt.svt_token_logprobs_backward(Stand(bf16, 4, 8), Stand(i64, 4), Stand(f32, 4), Stand(f32, 4), Stand(f32, 4)),
         "norms"),
        (lambda: svt.svt_token_logprobs_backward(Stand(bf16, 4, 8), Stand(i64, 4), Stand(f32, 4, 2), Stand(f32, 4),
                                                 Stand(bf16, 4)), "d_logprobs"),
        (lambda: svt.svt_gated_linear(Stand(bf16, 4, 8), Stand(bf16, 6, 7), Stand(bf16, 6, 8)), "w_gate"),
        (lambda: svt.svt_gated_linear(Stand(bf16, 4, 8), Stand(bf16, 6, 8), Stand(f32, 6, 8)), "w_up"),
        (lambda: svt.svt_gated_linear(Stand(bf16, 4, 8), Stand(bf16, 2, 6, 8), Stand(bf16, 2, 6, 8)), "w_gate"),
        (lambda: svt.svt_gated_linear(Stand(bf16, 4, 8), Stand(bf16, 2, 6, 8), Stand(bf16, 2, 6, 8), offsets=Stand(i32, 2)),
         "offsets"),
        (lambda: svt.svt_gated_linear(Stand(bf16, 4, 8), Stand(bf16, 6, 8), Stand(bf16, 6, 8), activation="tanh"),
         "activation"),
        (lambda: svt.svt_gated_linear_backward(Stand(bf16, 4, 5), Stand(bf16, 4, 8), Stand(bf16, 6, 8), Stand(bf16, 6, 8),
                                               Stand(bf16, 4, 6), Stand(bf16, 4, 6)), "dh"),
    ]
    for i, (call, name) in enumerate(bad):
        with pytest.raises(ValueError, match=name):
            call()
