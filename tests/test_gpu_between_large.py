"""Calls whose operands pass 2^31 elements: their last rows are those of a call on these alone, bit for bit."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def fill(*shape, dtype=torch.bfloat16, seed=0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(seed))


def test_norm_of_many_rows():
    rows, K, tail = 128 * 2100, 8192, 300
    x = fill(rows, K)
    assert x.numel() > 2 ** 31
    w = fill(K, dtype=torch.float32, seed=1)
    *whole, _, _ = mxq.mxq_rms_norm_fp8_group128_row_col(x, w)
    *last, _, _ = mxq.mxq_rms_norm_fp8_group128_row_col(x[-tail // 128 * 128:], w)
    n = last[0].shape[0]
    assert n == 384 and all(torch.equal(a[-b.shape[0]:], b) for a, b in zip(whole, last))
    del whole
    dy = fill(rows, K, seed=2)
    dx, dw = mxq.mxq_rms_norm_backward(dy, x, w)
    part, _ = mxq.mxq_rms_norm_backward(dy[-5:], x[-5:], w)
    assert torch.equal(dx[-5:], part)
    # the weight's gradient against sums of 64 bits over a few columns; each of the additions of up to rows values may be off by
    # half a step of the sum of magnitudes
    c = torch.tensor([0, 4097, K - 1], device=DEV)
    r = torch.cat([torch.rsqrt(p.float().square().mean(1).double() + 1e-6) for p in x.split(16384)])
    terms = dy[:, c].double() * x[:, c].double() * r[:, None]
    assert bool(((dw[c].double() - terms.sum(0)).abs() <= terms.abs().sum(0) * rows * 2.0 ** -24).all())


def test_activation_of_many_rows():
    rows, F = 128 * 1100, 16384
    h = fill(rows, 2 * F)
    whole = mxq.mxq_activate_fp8_group128_row_col(h[:, :F], h[:, F:])
    last = mxq.mxq_activate_fp8_group128_row_col(h[-256:, :F], h[-256:, F:])
    assert whole[0].numel() > 2 ** 31 and all(torch.equal(a[-b.shape[0]:], b) for a, b in zip(whole, last))
    row = mxq.mxq_activate_fp8_group128(h[:, :F], h[:, F:])
    assert torch.equal(row[0], whole[0]) and torch.equal(row[1], whole[1])
    del whole, row
    da = fill(rows, F, seed=1)
    whole = mxq.mxq_activate_fp8_group128_backward(da, h[:, :F], h[:, F:])
    last = mxq.mxq_activate_fp8_group128_backward(da[-256:], h[-256:, :F], h[-256:, F:])
    assert all(torch.equal(a[-b.shape[0]:], b) for a, b in zip(whole, last))


def test_route_of_many_tokens():
    tokens, E = 4_300_000, 512
    l = fill(tokens, E, dtype=torch.float32)
    assert l.numel() > 2 ** 31
    bias = fill(E, dtype=torch.float32, seed=1) * 0.1
    how = dict(bias=bias, score="sigmoid", n_groups=8, top_groups=4, group_top=2)
    ids, w = mxq.mxq_route_experts(l, 8, **how)
    some, part = mxq.mxq_route_experts(l[-1000:], 8, **how)
    assert torch.equal(ids[-1000:], some) and torch.equal(w[-1000:], part)
    d = mxq.mxq_route_experts_backward(w, l, ids, score="softmax", renormalize=False)
    part = mxq.mxq_route_experts_backward(w[-1000:], l[-1000:], ids[-1000:], score="softmax", renormalize=False)
    assert torch.equal(d[-1000:], part)
