"""Routed-expert entry points: every documented refusal, on the host (nothing is enqueued: the pointers are
never read), and the binding's checks of tensors."""
import ctypes

import pytest

from int8_ivf_ann_amd import svt

P = [0x10000000 + (i << 28) for i in range(8)]   # disjoint, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(svt.LIB_PATH):
        from int8_ivf_ann_amd import build
        build.build()
    return svt.lib()


def weights(M=1, N=32, K=64, group=32, scale_type=svt.SVT_F16, has_zeros=0, packed=0x70000000, nbytes=1 << 28):
    return svt.svt_quant_weights(M, N, K, group, scale_type, has_zeros, packed, nbytes)


def refused(rc, code=svt.SVT_EINVAL, text=None):
    assert rc == code, (rc, svt.svt_last_error())
    msg = svt.svt_last_error()
    assert msg and (text is None or text in msg), msg


BAD_ROUTE = [
    (dict(T=-1), "n_tokens"), (dict(E=0), "n_experts"), (dict(E=513), "n_experts"), (dict(top=0), "top"),
    (dict(top=17), "top"), (dict(E=4, top=5), "top"), (dict(dtype=3), "type"), (dict(dtype=-1), "type"),
    (dict(renorm=2), "renormalise"), (dict(a=None), "NULL"), (dict(b=None), "NULL"), (dict(c=None), "NULL"),
    (dict(a=P[0] + 2), "misaligned"), (dict(b=P[1] + 2), "misaligned"), (dict(c=P[2] + 1), "misaligned"),
    (dict(b=P[0] + 8), "overlap"), (dict(c=P[1]), "overlap"),
]


@pytest.mark.parametrize("kw, text", BAD_ROUTE)
def test_route_refusals(L, kw, text):
    v = dict(T=4, E=8, top=2, dtype=svt.SVT_F32, renorm=1, a=P[0], b=P[1], c=P[2])
    v.update(kw)
    refused(L.svt_route(v["T"], v["E"], v["top"], v["dtype"], v["a"], v["renorm"], v["b"], v["c"], None), text=text)


@pytest.mark.parametrize("kw, text", [
    (dict(T=-1), "n_tokens"), (dict(E=513), "n_experts"), (dict(top=9), "top"), (dict(dtype=7), "type"),
    (dict(renorm=-1), "renormalise"), *[(dict([(i, None)]), "NULL") for i in range(5)],
    (dict([(0, P[0] + 1)]), "misaligned"), (dict([(4, P[4] + 1)]), "misaligned"), (dict([(1, P[1] + 2)]), "misaligned"),
    (dict([(4, P[0])]), "overlap"), (dict([(4, P[3] + 4)]), "overlap"),
])
def test_route_backward_refusals(L, kw, text):
    v = dict(T=4, E=8, top=2, dtype=svt.SVT_BF16, renorm=0)
    v.update({i: P[i] for i in range(5)})
    v.update(kw)
    refused(L.svt_route_backward(v["T"], v["E"], v["top"], v["dtype"], v[0], v["renorm"], v[1], v[2], v[3], v[4], None),
            text=text)


@pytest.mark.parametrize("kw, text", [
    (dict(T=-1), "n_tokens"), (dict(top=0), "top"), (dict(top=17), "top"), (dict(E=0), "n_experts"),
    (dict(E=513), "n_experts"), (dict(T=2 ** 27, top=16), "2^30"), *[(dict([(i, None)]), "NULL") for i in range(4)],
    *[(dict([(i, P[i] + 2)]), "misaligned") for i in range(4)], (dict(ws=P[5] + 2), "misaligned"),
    (dict(T=100000, ws=None), "workspace"), (dict(T=100000, nb=64), "workspace"),
    (dict([(3, P[0])]), "overlap"), (dict([(1, P[2] + 16)]), "overlap"), (dict(T=100000, ws=P[3] + 64), "overlap"),
])
def test_sort_refusals(L, kw, text):
    v = dict(T=64, top=2, E=8, ws=P[5], nb=1 << 20)
    v.update({i: P[i] for i in range(4)})
    v.update(kw)
    refused(L.svt_expert_sort(v["T"], v["top"], v["E"], v[0], v[1], v[2], v[3], v["ws"], v["nb"], None), text=text)


def test_sort_workspace_size(L):
    assert L.svt_expert_sort_workspace_size(8, 2, 8) == 0 and not svt.svt_last_error()
    assert L.svt_expert_sort_workspace_size(1 << 20, 2, 64) > 0
    assert L.svt_expert_sort_workspace_size(1 << 26, 16, 512) < 1 << 24
    for bad in ((-1, 2, 8), (8, 0, 8), (8, 17, 8), (8, 2, 0), (8, 2, 513), (2 ** 27, 16, 8)):
        assert L.svt_expert_sort_workspace_size(*bad) == 0 and svt.svt_last_error()
        with pytest.raises(svt.SvtError):
            svt.svt_expert_sort_workspace_size(*bad)
    assert svt.svt_expert_sort_workspace_size(8, 2, 8) == 0


COMMON = [(dict(T=-1), "n_tokens"), (dict(top=0), "top"), (dict(top=17), "top"), (dict(T=2 ** 27, top=16), "2^30"),
          (dict(D=0), "width"), (dict(D=2 ** 24 + 1), "width"), (dict(dtype=3), "type")]


@pytest.mark.parametrize("kw, text", COMMON + [
    *[(dict([(i, None)]), "NULL") for i in range(3)], *[(dict([(i, P[i] + 1)]), "misaligned") for i in range(3)],
    (dict([(2, P[0] + 64)]), "overlap"), (dict([(2, P[1])]), "overlap")])
@pytest.mark.parametrize("name", ["svt_expert_dispatch", "svt_expert_dispatch_backward", "svt_expert_combine"])
def test_exchange_refusals(L, name, kw, text):
    v = dict(T=4, top=2, D=24, dtype=svt.SVT_F16)
    v.update({i: P[i] for i in range(3)})
    v.update(kw)
    extra = (P[6],) if name == "svt_expert_combine" else ()
    refused(getattr(L, name)(v["T"], v["top"], v["D"], v["dtype"], v[0], v[1], *extra, v[2], None), text=text)


@pytest.mark.parametrize("kw, text", COMMON + [
    *[(dict([(i, None)]), "NULL") for i in range(6)], *[(dict([(i, P[i] + 1)]), "misaligned") for i in range(6)],
    (dict([(4, P[1])]), "overlap"), (dict([(5, P[3])]), "overlap"), (dict([(5, P[4] + 8)]), "overlap")])
def test_combine_backward_refusals(L, kw, text):
    v = dict(T=4, top=2, D=24, dtype=svt.SVT_BF16)
    v.update({i: P[i] for i in range(6)})
    v.update(kw)
    refused(L.svt_expert_combine_backward(v["T"], v["top"], v["D"], v["dtype"], v[0], v[1], v[2], v[3], v[4], v[5],
                                          None), text=text)


BAD_WEIGHTS = [(dict(M=0), svt.SVT_EINVAL, "n_matrices"), (dict(M=513), svt.SVT_EINVAL, "n_matrices"),
               (dict(N=0), svt.SVT_EINVAL, "n_out"), (dict(N=2 ** 19 + 1), svt.SVT_EINVAL, "n_out"),
               (dict(K=0), svt.SVT_EINVAL, "n_in"), (dict(K=2 ** 20 + 1), svt.SVT_EINVAL, "n_in"),
               (dict(group=16), svt.SVT_EUNSUPPORTED, "group"), (dict(group=0), svt.SVT_EUNSUPPORTED, "group"),
               (dict(scale_type=3), svt.SVT_EINVAL, "scale type"), (dict(has_zeros=2), svt.SVT_EINVAL, "has_zeros")]


@pytest.mark.parametrize("kw, code, text", BAD_WEIGHTS)
def test_weights_refusals(L, kw, code, text):
    w = ctypes.byref(weights(**kw))
    assert L.svt_quant_pack_size(w) == 0 and text in svt.svt_last_error()
    refused(L.svt_quant_pack(w, P[0], P[1], None, None), code, text)
    refused(L.svt_quant_linear(4, svt.SVT_F16, P[0], w, P[1], None, 0, svt.SVT_F16, P[2], None), code, text)


@pytest.mark.parametrize("kw, args, text", [
    (dict(packed=None), {}, "NULL"), ({}, {0: None}, "NULL"), ({}, {1: None}, "NULL"), (dict(has_zeros=1), {}, "NULL"),
    ({}, {2: P[2]}, "zeros given"), (dict(nbytes=1024), {}, "packed buffer"), (dict(packed=0x70000080), {}, "misaligned"),
    ({}, {1: P[1] + 1}, "misaligned"), ({}, {0: 0x70000010}, "overlap"), ({}, {1: 0x70000010}, "overlap")])
def test_pack_refusals(L, kw, args, text):
    a = {0: P[0], 1: P[1], 2: None}
    a.update(args)
    refused(L.svt_quant_pack(ctypes.byref(weights(**kw)), a[0], a[1], a[2], None), text=text)


def test_null_weights(L):
    assert L.svt_quant_pack_size(None) == 0 and "NULL" in svt.svt_last_error()
    refused(L.svt_quant_pack(None, P[0], P[1], None, None), text="NULL")
    refused(L.svt_quant_linear(4, 0, P[0], None, None, None, 0, 0, P[2], None), text="NULL")


@pytest.mark.parametrize("kw, args, text", [
    ({}, dict(R=-1), "n_rows"), ({}, dict(dtype=9), "type"), ({}, dict(out=svt.SVT_BF16), "output type"),
    ({}, dict(out=5), "output type"), ({}, dict(act=2), "activation"), ({}, dict(act=-1), "activation"),
    (dict(M=2), dict(off=None), "offsets"), ({}, dict(x=None), "NULL"), ({}, dict(y=None), "NULL"),
    (dict(packed=None), {}, "NULL"), (dict(nbytes=100), {}, "packed buffer"), ({}, dict(x=P[0] + 1), "misaligned"),
    ({}, dict(y=P[2] + 1), "misaligned"), ({}, dict(off=P[1] + 2), "misaligned"), ({}, dict(bias=P[3] + 2), "misaligned"),
    (dict(packed=0x70000040), {}, "misaligned"), ({}, dict(y=P[0] + 8), "overlap"), ({}, dict(y=P[1]), "overlap"),
    ({}, dict(y=P[3]), "overlap"), ({}, dict(y=0x70000100), "overlap")])
def test_linear_refusals(L, kw, args, text):
    a = dict(R=4, dtype=svt.SVT_F16, x=P[0], off=P[1], bias=P[3], act=0, out=svt.SVT_F16, y=P[2])
    a.update(args)
    refused(L.svt_quant_linear(a["R"], a["dtype"], a["x"], ctypes.byref(weights(**kw)), a["off"], a["bias"], a["act"],
                               a["out"], a["y"], None), text=text)


def test_nothing_to_do_returns_ok(L):
    assert L.svt_route(0, 8, 2, 0, None, 1, None, None, None) == svt.SVT_OK
    assert L.svt_route_backward(0, 8, 2, 0, None, 1, None, None, None, None, None) == svt.SVT_OK
    assert L.svt_expert_dispatch(0, 2, 8, 0, None, None, None, None) == svt.SVT_OK
    assert L.svt_expert_dispatch_backward(0, 2, 8, 0, None, None, None, None) == svt.SVT_OK
    assert L.svt_expert_combine(0, 2, 8, 0, None, None, None, None, None) == svt.SVT_OK
    assert L.svt_expert_combine_backward(0, 2, 8, 0, None, None, None, None, None, None, None) == svt.SVT_OK
    assert L.svt_quant_linear(0, 0, None, ctypes.byref(weights()), None, None, 0, 0, None, None) == svt.SVT_OK


def test_header_constants_and_struct():
    import os
    import re
    hdr = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "svt.h")).read()
    assert re.search(r"SVT_F32 = 0, SVT_F16 = 1, SVT_BF16 = 2", hdr)
    assert re.search(r"SVT_ACT_NONE = 0, SVT_ACT_RELU = 1", hdr)
    assert re.search(rf"#define SVT_MAX_EXPERTS {svt.SVT_MAX_EXPERTS}\b", hdr)
    assert re.search(rf"#define SVT_MAX_TOP {svt.SVT_MAX_TOP}\b", hdr)
    assert re.search(r"int32_t n_matrices, n_out, n_in, group, scale_type, has_zeros;\s*void \*packed;\s*"
                     r"size_t packed_bytes;\s*\} svt_quant_weights;", hdr)
    assert [f[0] for f in svt.svt_quant_weights._fields_] == ["n_matrices", "n_out", "n_in", "group", "scale_type",
                                                              "has_zeros", "packed", "packed_bytes"]
    assert ctypes.sizeof(svt.svt_quant_weights) == 24 + ctypes.sizeof(ctypes.c_void_p) + ctypes.sizeof(ctypes.c_size_t)


def test_binding_refusals():
    """Host tensors, wrong shapes, types and layouts raise ValueError before the library is called."""
    import torch
    f = torch.zeros((4, 8))
    i = torch.zeros((4, 2), dtype=torch.int32)
    for call, text in [
        (lambda: svt.svt_route(f, 2), "device tensor"),
        (lambda: svt.svt_route(f[0], 2), "2-D"),
        (lambda: svt.svt_route(f.double(), 2), "dtype"),
        (lambda: svt.svt_route(f.t(), 2), "contiguous"),
        (lambda: svt.svt_route(None, 2), "2-D"),
        (lambda: svt.svt_route_backward(f, i, f, f), "device tensor"),
        (lambda: svt.svt_expert_sort(i.long(), 4), "dtype"),
        (lambda: svt.svt_expert_sort(i, 4), "device tensor"),
        (lambda: svt.svt_expert_sort(i[0], 4), "2-D"),
        (lambda: svt.svt_expert_sort(i.t(), 4), "contiguous"),
        (lambda: svt.svt_expert_dispatch(f, i), "device tensor"),
        (lambda: svt.svt_expert_combine(f.to(torch.int32), i), "dtype"),
        (lambda: svt.svt_expert_combine_backward(f, f, i, f), "device tensor"),
        (lambda: svt.svt_expert_dispatch_backward(f, i), "device tensor"),
        (lambda: svt.svt_quant_pack(i[None], f, None, 8, 32), "3-D"),
        (lambda: svt.svt_quant_linear(f, weights()), "device tensor"),
    ]:
        with pytest.raises(ValueError, match=text):
            call()


def test_calls_run_on_the_tensors_device(monkeypatch):
    """Tensors of another device than the current one: the call makes that device current and takes its stream;
    a stream of another device is refused.  (Without devices: torch's functions are stood in for.)"""
    import torch
    entered = []

    class Guard:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            entered.append(self.what)

        def __exit__(self, *exc):
            entered.append(("left", self.what))

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 77

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: Guard(("device", d.index)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: Guard(("stream", s.cuda_stream)))
    monkeypatch.setattr(svt, "_raw_stream", lambda index: 1000 + index)
    with svt._Run(torch.device("cuda", 1), None) as handle:
        assert handle == 1001 and entered == [("device", 1)]
    assert entered == [("device", 1), ("left", ("device", 1))]
    del entered[:]
    with svt._Run(torch.device("cuda", 0), None) as handle:
        assert handle == 1000 and entered == []
    with svt._Run(torch.device("cuda", 1), Stream) as handle:
        assert handle == 77 and entered == [("stream", 77)]
    with pytest.raises(ValueError, match="stream"):
        svt._Run(torch.device("cuda", 0), Stream)
