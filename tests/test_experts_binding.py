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
