"""The activation with FP8 output and its gradients against 64-bit forms: every activation, with
and without a second half, odd sizes, strides and alignments, rows by expert with empty experts and rows of
none, tails, values that are not finite, captured."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import between_ref as ref
from tests.test_gpu_products import odd_view

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
ACTS = ("silu", "gelu_tanh", "relu2")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def values(rows, cols, g, dtype, spread=3):
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (rows, 1), generator=g).float())
    if rows > 2:
        x[1] = 0
    return x.to(dtype)


def check(rows, F, act, gated, dtype, place, seed, offsets=None):
    g = gen(seed)
    h, da = values(rows, 2 * F if gated else F, g, dtype), values(rows, F, g, dtype)
    hd, dad = place(h), place(da)
    gate, up = (hd[:, :F], hd[:, F:]) if gated else (hd, None)
    hg, hu = (h[:, :F], h[:, F:]) if gated else (h, None)
    od = None if offsets is None else offsets.to(DEV)
    want, off = ref.activate(act, hg, hu)
    q, c = mxq.mxq_activate_fp8_group128(gate, up, act)
    ref.check_rows(q, c, want, off)
    rq, rc, cq, cc = mxq.mxq_activate_fp8_group128_row_col(gate, up, act, offsets=od)
    if offsets is None:
        assert torch.equal(rq, q) and torch.equal(rc, c)
    ref.check_rows(rq, rc, want, off)
    ref.check_cols(cq, cc, want, off, offsets)
    want, off = ref.activate_backward(act, da, hg, hu)
    rq, rc, cq, cc = mxq.mxq_activate_fp8_group128_backward(dad, gate, up, act, offsets=od)
    ref.check_rows(rq, rc, want, off, "gradient rows")
    ref.check_cols(cq, cc, want, off, offsets, "gradient columns")


SIZES = [(1, 1), (1, 128), (2, 3), (3, 130), (16, 256), (54, 1024), (130, 136), (257, 40), (128, 1000), (5, 100), (9, 203)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("rows,F", SIZES)
def test_activation_sizes(rows, F, gated, dtype):
    act = ACTS[(rows + F) % 3]
    check(rows, F, act, gated, dtype, lambda t: t.to(DEV), rows + F)
    check(rows, F, "silu", gated, dtype, odd_view, rows + F + 1)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("F", [256, 264, 250])
@pytest.mark.parametrize("offsets", [[0, 0, 5, 135, 135, 300], [10, 20, 20, 290], [0, 400, 100, 5000, -3, 280], [0, 0, 0], [0, 301]])
def test_activation_by_expert(act, F, offsets):
    """Empty experts, rows of none before and behind, offsets that fall or leave the matrix."""
    check(301, F, act, True, BF16, lambda t: t.to(DEV), F, torch.tensor(offsets, dtype=torch.int32))
    check(301, F, act, False, FP32, lambda t: t.to(DEV), F, torch.tensor(offsets, dtype=torch.int32))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_activation_tails(act, dtype):
    """Far out in both directions, at zero and next to it: column groups of one row keep every value's own scale."""
    g = torch.cat([torch.linspace(-110, 110, 881), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-4, -1e-4, 1e4, -1e4, 3e18, -3e18])])
    g = g.to(dtype)[None]
    up, da = torch.full_like(g, 0.75), torch.full_like(g, -1.25)
    want, off = ref.activate(act, g, up)
    _, _, cq, cc = mxq.mxq_activate_fp8_group128_row_col(g.to(DEV), up.to(DEV), act)
    ref.check_cols(cq, cc, want, off)
    want, off = ref.activate_backward(act, da, g, up)
    _, _, cq, cc = mxq.mxq_activate_fp8_group128_backward(da.to(DEV), g.to(DEV), up.to(DEV), act)
    ref.check_cols(cq, cc, want, off)


@pytest.mark.parametrize("act", ACTS)
def test_activation_of_values_that_are_not_finite(act):
    """An Inf or NaN in either half poisons its groups and no others."""
    g = gen(7)
    h = torch.randn(140, 512, generator=g)
    for r, c, v in ((3, 5, float("nan")), (10, 200, float("inf")), (130, 256 + 7, float("nan")), (20, 256 + 130, float("inf"))):
        h[r, c] = v
    bad = ~torch.isfinite(h[:, :256] * h[:, 256:])
    for dtype in (BF16, FP32):
        v = h.to(dtype).to(DEV)
        q, c, cq, cc = (ref.host(t) for t in mxq.mxq_activate_fp8_group128_row_col(v[:, :256], v[:, 256:], act))
        poisoned = torch.stack([bad[:, :128].any(1), bad[:, 128:].any(1)], 1)
        assert torch.equal(c == 255, poisoned)
        assert bool((q.view(140, 2, 128)[poisoned] == 0x7F).all())
        columns = torch.stack([bad[:128].any(0), bad[128:].any(0)])
        assert torch.equal(cc == 255, columns)


def test_activation_across_the_ends_of_a_call():
    """Rows of [dgate, dup] whose groups straddle the halves, at every place of the border within eight columns."""
    for F in range(121, 137):
        check(20, F, "silu", True, BF16, lambda t: t.to(DEV), F)


def test_activation_leaves_the_rest_alone():
    h = torch.randn(6, 400, generator=gen(6)).to(DEV)
    bufs = [torch.full((9, 420), 9, dtype=torch.uint8, device=DEV) for _ in range(4)]
    views = [bufs[0][1:7, 3:203], bufs[1][1:7, 1:3], bufs[2][1:7, 3:203], bufs[3][1:2, 3:203]]
    mxq.mxq_activate_fp8_group128_row_col(h[:, :200], h[:, 200:], "silu", row_data=views[0], row_scale=views[1], col_data=views[2],
                                          col_scale=views[3])
    for b, v in zip(bufs, views):
        v.fill_(9)
        assert bool((b == 9).all())


def test_activation_captured():
    offsets = torch.tensor([0, 40, 40, 150], dtype=torch.int32, device=DEV)
    h, da = values(160, 512, gen(1), BF16).to(DEV), values(160, 256, gen(2), BF16).to(DEV)

    def step(h, da):
        return (*mxq.mxq_activate_fp8_group128(h[:, :256], h[:, 256:]),
                *mxq.mxq_activate_fp8_group128_row_col(h[:, :256], h[:, 256:], offsets=offsets),
                *mxq.mxq_activate_fp8_group128_backward(da, h[:, :256], h[:, 256:], offsets=offsets))

    step(h, da)
    sh, sd, so = h.clone(), da.clone(), offsets.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(sh, sd)
    for k in range(4):
        sh.copy_(h.roll(k, 0) * (k + 1))
        sd.copy_(da * (0.5 + k))
        offsets.copy_(torch.tensor([0, 40 + 11 * k, 60 + 11 * k, 150], dtype=torch.int32))
        want = step(sh, sd)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
    offsets.copy_(so)
