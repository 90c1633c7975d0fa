"""The gradient of rows that no slot names."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_a_padded_buffer_have_no_gradient(dtype):
    tokens, top_k, H, R = 40, 2, 256, 300
    rows, dy = torch.ones(R, H, dtype=dtype, device="cuda"), torch.ones(tokens, H, dtype=dtype, device="cuda")
    position = torch.arange(tokens * top_k, dtype=torch.int32, device="cuda").view(tokens, top_k) + 7
    used = torch.full((R, H), float("nan"), dtype=dtype, device="cuda")
    del used                                    # the next allocation of this size finds its bytes
    drows, dw = mxq.mxq_combine_rows_backward(dy, rows, position)
    named = torch.zeros(R, dtype=torch.bool, device="cuda")
    named[7:7 + tokens * top_k] = True
    assert (drows[named] == 1).all() and (drows[~named] == 0).all()
    given = torch.full((R, H), 5.0, dtype=dtype, device="cuda")
    mxq.mxq_combine_rows_backward(dy, rows, position, drows=given)
    assert (given[named] == 1).all() and (given[~named] == 5).all()
