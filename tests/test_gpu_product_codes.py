"""The FP8 products at codes and code strides out of the ordinary, at sizes that take
the many-rows kernels, against plain 64-bit forms (tests/fp8_ref.py has the tolerances)."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import fp8_ref as ref
from tests.test_gpu_products import DEV, codes, dev, gen, odd_view, payload

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


# Sizes of y (M x N), dx (M x N) and dw (M x N): y and dx have too many rows for the few-rows kernels.
SIZES = {"y": (512, 256, 4160), "dx": (512, 256, 4160), "dw": (300, 264, 272)}


def product_of(which, place, vq, vc, uq, uc, **kw):
    """which as V U^T on the device: vq [rows, R], uq [columns, R] and their codes, R blocks of 128 along columns
    (y, dx) -- laid out as each call takes them."""
    t = lambda a: place(a.t().contiguous())
    kw.setdefault("out_dtype", torch.float32)
    if which == "y":
        return mxq.mxq_matmul_fp8_block128(place(vq), place(vc), place(uq), place(uc), **kw)
    if which == "dx":
        return mxq.mxq_matmul_fp8_block128_dgrad(place(vq), place(vc), t(uq), t(uc), **kw)
    return mxq.mxq_matmul_fp8_group128_wgrad(t(vq), t(vc), t(uq), t(uc), **kw)


@pytest.mark.parametrize("place", [dev, odd_view])
@pytest.mark.parametrize("which", ["y", "dx", "dw"])
def test_products_that_cancel(which, place):
    """Each product has its negative beside it, so every sum is 0 whatever the codes.  Payloads are multiples of
    32, so that unscaled sums are exact in fp32."""
    I, R, J = SIZES[which]
    g = gen(31)
    coarse = lambda *s: torch.randint(-14, 15, s, generator=g).float() * 32
    a, b = coarse(I, R // 2), coarse(J, R // 2)
    a[0], b[0] = 448, 448
    q8 = lambda v: v.flatten(1).to(torch.float8_e4m3fn).view(torch.uint8)
    exact = lambda v: v.to(torch.float8_e4m3fn).float()
    a, b = exact(a), exact(b)
    vq, uq = q8(torch.stack([a, a], -1)), q8(torch.stack([b, -b], -1))
    one_code = lambda rows, c: torch.full((rows, ref.ceil_div(R)), c, dtype=torch.uint8)
    for cv, cu in ((167, 167), (168, 168), (190, 190), (246, 246), (254, 254), (246, 127), (77, 250)):
        uc = one_code(J if which == "dw" else ref.ceil_div(J), cu)
        out = product_of(which, place, vq, one_code(I, cv), uq, uc)
        assert (out == 0).all(), f"codes {cv} {cu}: {int(torch.isnan(out).sum())} NaN of {out.numel()}"
