"""The whole-block operators refuse tensors of other than two dimensions as they refuse any other argument.  No GPU needed."""

import pytest
import torch

import moe_grouped_gemm_block_gb300 as g

BF16, I32 = torch.bfloat16, torch.int32
SHAPES = [(), (8,), (2, 2, 8)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("call", [
    lambda t: g.moe_route(t, 2),
    lambda t: g.moe_route_backward(t, torch.zeros(2, 2, dtype=I32), torch.zeros(2, 2)),
    lambda t: g.residual_rms_norm(t),
    lambda t: g.residual_rms_norm(t, t, post_norm=True),
    lambda t: g.residual_rms_norm(torch.zeros(2, 8, dtype=BF16), t),
    lambda t: g.residual_rms_norm_backward(t, None, t, None, torch.zeros(2)),
    lambda t: g.residual_rms_norm_backward(t, t, torch.zeros(2, 8, dtype=BF16), t, torch.zeros(2)),
    lambda t: g.swiglu(t),
    lambda t: g.swiglu_quantize_1x128(t),
    lambda t: g.swiglu_backward(t, t),
    lambda t: g.swiglu_backward(t, t, keep=False),
    lambda t: g.swiglu_backward(t, torch.zeros(2, 16, dtype=BF16)),
])
def test_other_shapes_are_refused(call, shape):
    with pytest.raises(ValueError):
        call(torch.zeros(shape, dtype=BF16))
