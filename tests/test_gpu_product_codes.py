"""The FP8 products at codes and code strides out of the ordinary, at sizes that take
the many-rows kernels, against plain 64-bit forms (tests/fp8_ref.py has the tolerances)."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import fp8_ref as ref
from tests.test_gpu_products import DEV, codes, dev, gen, payload

pytestmark = pytest.mark.gpu


def far_apart(t, stride):
    """The same 2-D bytes on the device, rows `stride` bytes apart."""
    buf = torch.empty(t.shape[0] * stride, dtype=torch.uint8, device=DEV).view(t.shape[0], stride)[:, :t.shape[1]]
    buf.copy_(t)
    return buf


def test_codes_of_rows_far_apart():
    """Code rows 34.1 million bytes apart: 63 of them pass 2^31."""
    M, R, J, g = 128, 300, 16512, gen(21)
    vq, vc, wc = payload(g, M, R), codes(g, M, ref.ceil_div(R)), codes(g, ref.ceil_div(J), ref.ceil_div(R))
    wq, far = payload(g, J, R), far_apart(vc, 34_100_000)
    y = mxq.mxq_matmul_fp8_block128(dev(vq), far, dev(wq), dev(wc), out_dtype=torch.float32)
    ref.check(y, *ref.matmul(vq, vc, wq, wc), R, "y")
    wq, wc = wq.t().contiguous(), wc.t().contiguous()
    dx = mxq.mxq_matmul_fp8_block128_dgrad(dev(vq), far, dev(wq), dev(wc), out_dtype=torch.float32)
    ref.check(dx, *ref.matmul(vq, vc, wq, wc, transpose=True), R, "dx")
