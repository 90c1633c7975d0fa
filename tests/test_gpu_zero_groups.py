"""Groups of zeros in the products summed in fp32: their code is 0, any scale does for
them, and they cost no time."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import fp8_ref as ref
from tests.product_sizes import CASES
from tests.test_gpu_product_kernels import DEV, call, dev, expected, gen, odd, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [c for c in CASES if c.kernel.startswith("kExact")], ids=str)
@pytest.mark.parametrize("kind", ["some", "signed", "all"])
def test_zero_groups(c, kind):
    g = gen(c.I + c.R)
    v, vc, u, uc, offsets = operands(c, g)
    zero = 0x80 if kind == "signed" else 0
    rows = slice(None) if kind == "all" else slice(1, None, 7)
    if c.mode == "dw":                       # whole columns: every group of them, wherever an expert's begin
        v[:, rows], vc[:, rows] = zero, 0
        u[:, 3::11], uc[:, 3::11] = zero, 0
    else:
        v[rows, 128:256], vc[rows, 1] = zero, 0
        n = slice(128, 256)                  # one tile of each weight
        u[..., n, n], uc[..., 1, 1] = zero, 0
    out = call(c, dev if c.fed else odd, v, vc, u, uc, offsets, out_dtype=torch.float32)
    ref.check(out, *expected(c, v, vc, u, uc, offsets), c.R, f"{c} {kind}")


@pytest.mark.parametrize("c", [c for c in CASES if c.kernel.startswith("kExact")], ids=str)
def test_code_0_of_values_that_are_not_zero(c):
    """Code 0 beside zero groups of code 0: the values are 2^-127 of their payload, not 0."""
    v, vc, u, uc, offsets = operands(c, gen(c.J))
    blocks = vc if c.mode == "dw" else vc.t()
    blocks[0, ::2] = 0
    if c.mode == "dw":
        v[:, ::4] = 0
        v[5, ::4] = 0x38
    else:
        v[::4, :128] = 0
        v[::4, 77] = 0x38
    uc.fill_(167)
    out = call(c, dev if c.fed else odd, v, vc, u, uc, offsets, out_dtype=torch.float32)
    ref.check(out, *expected(c, v, vc, u, uc, offsets), c.R, str(c))


@pytest.mark.parametrize("which", ["y", "dx", "dw"])
def test_zero_groups_cost_no_time(which):
    """One zero group in each wave's first block against none: the way around took 4 times as long."""
    M, N, K = 4096, 2048, 2048
    g = torch.Generator(device=DEV).manual_seed(1)
    x, dy = torch.randn(M, K, generator=g, device=DEV), torch.randn(M, N, generator=g, device=DEV)
    w = mxq.mxq_mxfp4_to_fp8_block128((torch.randn(N, K, generator=g, device=DEV) * 0.02).bfloat16())

    def pass_of(zeros):
        a, b = x.clone(), dy.clone()
        if zeros:
            a[::32, :128] = 0
            b[::32, :128] = 0
            a[:128, ::32] = 0
        if which == "dw":
            ops = mxq.mxq_quantize_fp8_group128_col(b) + mxq.mxq_quantize_fp8_group128_col(a)
            return lambda: mxq.mxq_matmul_fp8_group128_wgrad(*ops)
        fn, ops = ((mxq.mxq_matmul_fp8_block128, mxq.mxq_quantize_fp8_group128(a)) if which == "y" else
                   (mxq.mxq_matmul_fp8_block128_dgrad, mxq.mxq_quantize_fp8_group128(b)))
        return lambda: fn(*ops, *w)

    def time(f):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b)

    dense, zeros = pass_of(False), pass_of(True)
    time(dense), time(zeros)
    took = sorted(time(zeros) / time(dense) for _ in range(5))
    assert took[2] < 2, took
