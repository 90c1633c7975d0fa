"""Calls by expert on no rows at all (an empty batch): every code row is one that no group needs, and those are 0."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def codes(K):
    """A code array inside a larger one, and whether the rest of that still holds what it held."""
    buf = torch.full((7, K + 9), 9, dtype=torch.uint8, device=DEV)
    view = buf[1:6, 3:3 + K]

    def rest_is_left():
        around = torch.ones_like(buf, dtype=torch.bool)
        around[1:6, 3:3 + K] = False
        return bool((buf[around] == 9).all())
    return view, rest_is_left


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("F", [1, 40, 128, 200, 1024])
def test_no_rows_by_expert(F, dtype):
    x, none = torch.zeros(0, F, dtype=dtype, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    full = torch.ones(5, F, dtype=dtype, device=DEV)
    for offsets in ([0, 0, 0, 0, 0, 0], [3, 9, -4, 2 ** 30, 0, 7]):     # clamped to the rows that there are
        o = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        for K, call in ((F, lambda c: mxq.mxq_quantize_fp8_group128_col(x, offsets=o, scale=c)),
                        (F, lambda c: mxq.mxq_quantize_fp8_group128_row_col(x, offsets=o, col_scale=c)),
                        (F, lambda c: mxq.mxq_quantize_fp8_group128_row_col(full, none, 2, offsets=o, col_scale=c)),
                        (F, lambda c: mxq.mxq_activate_fp8_group128_row_col(x, x, offsets=o, col_scale=c)),
                        (F, lambda c: mxq.mxq_activate_fp8_group128_row_col(x, offsets=o, col_scale=c)),
                        (2 * F, lambda c: mxq.mxq_activate_fp8_group128_backward(x, x, x, offsets=o, col_scale=c)),
                        (F, lambda c: mxq.mxq_activate_fp8_group128_backward(x, x, offsets=o, col_scale=c))):
            c, rest_is_left = codes(K)
            call(c)
            assert bool((c == 0).all()) and rest_is_left()
    assert mxq.mxq_activate_fp8_group128_row_col(x, x)[3].shape == (0, F)
