"""The binding of the routed-expert entry points, without a device: what it refuses before the library is called."""
import pytest

from int8_ivf_ann_amd import svt


def test_tensors_that_require_grad_are_refused():
    """No call records history: where torch would, a tensor that requires grad is refused, not silently cut off."""
    import torch
    f = torch.zeros((4, 8), requires_grad=True)
    i = torch.zeros((4, 2), dtype=torch.int32)
    calls = [lambda: svt.svt_route(f, 2), lambda: svt.svt_route_backward(f, i, f, f),
             lambda: svt.svt_expert_dispatch(f, i), lambda: svt.svt_expert_dispatch_backward(f, i),
             lambda: svt.svt_expert_combine(f, i), lambda: svt.svt_expert_combine_backward(f, f, i, f),
             lambda: svt.svt_quant_pack(i[None], f[None], None, 8, 32),
             lambda: svt.svt_quant_linear(f, svt.svt_quant_weights())]
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):   # the next check
            call()


class Stand:
    """A device tensor's attributes, without a device or storage."""
    is_cuda, requires_grad = True, False

    def __init__(self, dtype, *shape):
        import torch
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000


def test_router_takes_more_entries_than_the_sort(monkeypatch):
    """2^31 entries (the sort and the exchange stop at 2^30): what svt_route returns, its gradient takes."""
    import contextlib
    import torch
    T, E, K = 2 ** 27, 16, 16
    seen = []
    library = type("L", (), {n: (lambda *a, n=n: seen.append((n, a[:3])) or svt.SVT_OK)
                             for n in ("svt_route", "svt_route_backward")})
    monkeypatch.setattr(svt, "lib", lambda: library)
    monkeypatch.setattr(svt, "_Run", lambda dev, stream: contextlib.nullcontext(0))
    l, ids, w = Stand(torch.bfloat16, T, E), Stand(torch.int32, T, K), Stand(torch.float32, T, K)
    svt.svt_route(l, K, out_experts=ids, out_weights=w)
    svt.svt_route_backward(l, ids, w, w, out=l)
    assert seen == [("svt_route", (T, E, K)), ("svt_route_backward", (T, E, K))]
    for bad in (Stand(torch.int32, T - 1, K), Stand(torch.int64, T, K), Stand(torch.int32, T)):
        with pytest.raises(ValueError, match="experts"):
            svt.svt_route_backward(l, bad, w, w, out=l)
    with pytest.raises(ValueError, match="2\\^30"):
        svt.svt_expert_sort(ids, E)
