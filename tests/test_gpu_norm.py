"""The norm with the residual's addition and FP8 output, and its gradients, against 64-bit
forms: every way that a row is held, odd sizes, strides and alignments, types, rows that are zero, huge or
not finite, in place, captured, on another stream."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import between_ref as ref
from tests.test_gpu_products import odd_view

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
EPS = 1e-5


def gen(seed):
    return torch.Generator().manual_seed(seed)


def values(rows, K, g, dtype, spread=6):
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (rows, 1), generator=g).float())
    x[:, torch.rand(K, generator=g) < 0.02] *= 16
    if rows > 2:
        x[rows // 2] = 0
    return x.to(dtype)


def check_norm(rows, K, dtype, stream, with_res, w_dtype, place, seed, cols):
    g = gen(seed)
    x, res = values(rows, K, g, dtype), values(rows, K, g, stream) if with_res else None
    w = None if w_dtype is None else (1 + 0.2 * torch.randn(K, generator=g)).to(w_dtype)
    s = ref.stored_sum(x, res)
    want, off = ref.norm(s, w, EPS)
    xd, rd = place(x), None if res is None else place(res)
    wd = None if w is None else w.to(DEV)
    y, got = mxq.mxq_rms_norm(xd, wd, EPS, residual=rd)
    ref.check_values(y, want, off, "y")
    if with_res:
        assert got.dtype == stream and torch.equal(ref.f64(got), s), "sum"
    else:
        assert got is None
    q, c, got, y2 = mxq.mxq_rms_norm_fp8_group128(xd, wd, EPS, residual=rd, with_y=True)
    ref.check_rows(q, c, want, off)
    assert torch.equal(y2, y) and (not with_res or torch.equal(ref.f64(got), s))
    q2, c2, _, none = mxq.mxq_rms_norm_fp8_group128(xd, wd, EPS, residual=rd)
    assert none is None and torch.equal(q2, q) and torch.equal(c2, c)
    if cols:
        rq, rc, cq, cc, got, y3 = mxq.mxq_rms_norm_fp8_group128_row_col(xd, wd, EPS, residual=rd, with_y=True)
        assert torch.equal(rq, q) and torch.equal(rc, c) and torch.equal(y3, y)
        assert not with_res or torch.equal(ref.f64(got), s)
        ref.check_cols(cq, cc, want, off)


# every number of lanes and pieces that a row takes, and its borders
WIDTHS = [1, 7, 8, 127, 128, 129, 512, 520, 1000, 2048, 2049, 2056, 4096, 4104, 5120, 5128, 6000, 6144, 6152, 8191, 8192, 8200, 16384, 16385, 16400, 20000]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("K", WIDTHS)
def test_norm_widths(K, dtype):
    check_norm(5, K, dtype, dtype, True, dtype, lambda t: t.to(DEV), K, K <= 4104)
    check_norm(3, K, dtype, dtype, True, FP32, odd_view, K + 1, K <= 1000)


@pytest.mark.parametrize("rows,K", [(1, 8192), (2, 130), (17, 96), (128, 256), (129, 136), (300, 72), (700, 264), (1025, 640)])
@pytest.mark.parametrize("dtype,stream", [(BF16, BF16), (BF16, FP32), (FP32, FP32), (FP32, BF16)])
def test_norm_types(rows, K, dtype, stream):
    check_norm(rows, K, dtype, stream, True, BF16, lambda t: t.to(DEV), rows + K, True)
    check_norm(rows, K, dtype, dtype, False, None, lambda t: t.to(DEV), rows + K + 1, True)


def test_norm_many_short_rows():
    check_norm(4000, 128, BF16, BF16, False, BF16, lambda t: t.to(DEV), 1, False)
    check_norm(2500, 64, FP32, FP32, True, FP32, lambda t: t.to(DEV), 2, False)


@pytest.mark.parametrize("K", [100, 1000, 8192, 20000])
def test_norm_in_place(K):
    """The sum where the residual was; y and the payload are those of a call with a place of its own for it."""
    g = gen(K)
    x, res, w = values(9, K, g, BF16).to(DEV), values(9, K, g, FP32).to(DEV), torch.randn(K, generator=g).to(DEV)
    want = mxq.mxq_rms_norm_fp8_group128(x, w, EPS, residual=res, with_y=True)
    for fn in (mxq.mxq_rms_norm_fp8_group128, mxq.mxq_rms_norm_fp8_group128_row_col):
        r = res.clone()
        out = fn(x, w, EPS, residual=r, residual_out=r, with_y=True)
        assert out[-2] is r and torch.equal(r, want[2])
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(out[-1], want[3])
    # run again from the stored sum: the same bits, without the addition
    again = mxq.mxq_rms_norm_fp8_group128(want[2], w, EPS)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_norm_columns_without_a_stored_sum():
    """The C call may leave the sum out: the columns then come from x and the residual."""
    g = gen(4)
    x, res, w = values(150, 264, g, BF16).to(DEV), values(150, 264, g, BF16).to(DEV), torch.randn(264, generator=g).to(DEV)
    want = mxq.mxq_rms_norm_fp8_group128_row_col(x, w, EPS, residual=res)
    L = mxq.load()
    outs = [torch.zeros_like(t) for t in want[:4]]
    ws = torch.empty(L.mxq_rms_norm_fp8_group128_row_col_workspace(150), dtype=torch.uint8, device=DEV)
    rc = L.mxq_rms_norm_fp8_group128_row_col(x.data_ptr(), 264, res.data_ptr(), 264, 0, w.data_ptr(), 1, EPS, 150, 264, 0, None, 0,
                                             None, 0, outs[0].data_ptr(), 264, outs[1].data_ptr(), 3, outs[2].data_ptr(), 264,
                                             outs[3].data_ptr(), 264, ws.data_ptr(), ws.numel(), mxq._handle(x))
    assert rc == mxq.MXQ_OK
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("K", [96, 400, 3000, 20000])
def test_norm_extremes(K):
    """Squares that overflow or vanish, rows with one Inf or NaN: the formula's values."""
    g = gen(K)
    x = torch.randn(7, K, generator=g)
    x[0] *= 1e30
    x[1] = 3.3e38
    x[2] *= 1e-30
    x[3, K // 2] = float("inf")
    x[4, K - 1] = float("nan")
    x[5] *= torch.exp2(torch.randint(-120, 120, (K,), generator=g).float())
    for dtype in (FP32, BF16):
        v = x.to(dtype)
        s = ref.f64(v)
        want, off = ref.norm(s, None, EPS)
        row = torch.where(torch.isinf(s[3]), torch.nan, 0.0)
        want[3], off[3] = row, 0.0
        y, _ = mxq.mxq_rms_norm(v.to(DEV), None, EPS)
        # values far below the row's largest: 2^-149 of an fp32 step
        ref.check_values(y, want, off + 2.0 ** -147, "y")
        q, c, _, _ = mxq.mxq_rms_norm_fp8_group128(v.to(DEV), None, EPS)
        ref.check_rows(q, c, want, off + 2.0 ** -147)


def check_backward(rows, K, dtype, x_dtype, w_dtype, with_res, place, seed):
    g = gen(seed)
    x, dy = values(rows, K, g, x_dtype), values(rows, K, g, dtype, 2)
    res = values(rows, K, g, x_dtype, 2) if with_res else None
    w = None if w_dtype is None else (1 + 0.2 * torch.randn(K, generator=g)).to(w_dtype)
    (dx, dx_off), (dw, dw_off) = ref.norm_backward(dy, ref.f64(x), w, EPS, res)
    got, got_w = mxq.mxq_rms_norm_backward(place(dy), place(x), None if w is None else w.to(DEV), EPS,
                                           dresidual=None if res is None else place(res))
    assert got.dtype == x_dtype and got_w.dtype == FP32
    ref.check_values(got, dx, dx_off, "dx")
    ref.check_values(got_w, dw, dw_off, "dweight")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("K", WIDTHS)
def test_norm_backward_widths(K, dtype):
    check_backward(5, K, dtype, dtype, dtype, True, lambda t: t.to(DEV), K)
    check_backward(3, K, dtype, dtype, FP32, True, odd_view, K + 1)


@pytest.mark.parametrize("rows,K", [(1, 8192), (2, 130), (17, 96), (256, 264), (257, 72), (1500, 128), (1100, 2056)])
@pytest.mark.parametrize("dtype,x_dtype", [(BF16, BF16), (BF16, FP32), (FP32, FP32), (FP32, BF16)])
def test_norm_backward_types(rows, K, dtype, x_dtype):
    check_backward(rows, K, dtype, x_dtype, BF16, True, lambda t: t.to(DEV), rows + K)
    check_backward(rows, K, dtype, x_dtype, None, False, lambda t: t.to(DEV), rows + K + 1)


@pytest.mark.parametrize("K", [96, 400, 3000, 20000])
def test_norm_backward_extremes(K):
    """Squares that overflow in some rows and not in their neighbours; a row of an Inf or NaN spoils dx of its own alone."""
    g = gen(K)
    x, dy = torch.randn(9, K, generator=g), torch.randn(9, K, generator=g)
    x[0] *= 1e30
    x[3] = 3.3e38
    x[4] *= 1e25
    x[6] *= 1e-30
    for dtype in (FP32, BF16):
        v, d = x.to(dtype), dy.to(dtype)
        (dx, dx_off), (dw, dw_off) = ref.norm_backward(d, ref.f64(v), None, EPS, None)
        got, got_w = mxq.mxq_rms_norm_backward(d.to(DEV), v.to(DEV), None, EPS)
        # r of the second row is below 2^-126 and has 20 places or more
        ref.check_values(got, dx, dx_off + dx.abs() * 2.0 ** -20 + 2.0 ** -147, "dx")
        ref.check_values(got_w, dw, dw_off + dy.abs().sum(0).double() * 2.0 ** -20, "dweight")
        v[4, 5], v[8, K - 1] = float("inf"), float("nan")
        spoilt, _ = mxq.mxq_rms_norm_backward(d.to(DEV), v.to(DEV), None, EPS)
        keep = [r for r in range(9) if r not in (4, 8)]
        assert torch.equal(spoilt[keep], got[keep]) and bool(torch.isnan(spoilt[8]).all())


@pytest.mark.parametrize("K", [96, 400, 3000, 20000])
def test_norm_backward_of_large_gradients(K):
    """Rows whose sum of g s passes 2^128, with and without the sum of squares, where dx does not."""
    g = gen(K + 1)
    x, dy = torch.randn(5, K, generator=g), torch.randn(5, K, generator=g)
    x[0] *= 1e4
    x[2] *= 1e30
    dy[0] *= 1e36
    dy[2] *= 1e36
    dy[3] *= 1e36
    for dtype in (FP32, BF16):
        v, d = x.to(dtype), dy.to(dtype)
        (dx, dx_off), (dw, dw_off) = ref.norm_backward(d, ref.f64(v), None, EPS, None)
        got, got_w = mxq.mxq_rms_norm_backward(d.to(DEV), v.to(DEV), None, EPS)
        ref.check_values(got, dx, dx_off + 2.0 ** -147, "dx")
        ref.check_values(got_w, dw, dw_off, "dweight")


def test_norm_backward_against_differences():
    """dx and dweight against differences of the forward call itself: f = <y, dy> moved by a step along a direction.  With
    fp32 values of about 1 a difference of two sums of n = 80 products is off by 2 n 2^-24 |terms| / (2 h), h = 2^-6, and by
    h^2 of the third derivative."""
    g = gen(8)
    x, w, dy = torch.randn(2, 40, generator=g), 1 + 0.2 * torch.randn(40, generator=g), torch.randn(2, 40, generator=g)
    dx, dw = mxq.mxq_rms_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), EPS)
    f = lambda x, w: float((ref.f64(mxq.mxq_rms_norm(x.to(DEV), w.to(DEV), EPS)[0]) * dy.double()).sum())
    h = 2.0 ** -6
    for k in range(4):
        v = torch.randn(2, 40, generator=g)
        v /= v.norm()
        got = (f(x + h * v, w) - f(x - h * v, w)) / (2 * h)
        assert abs(got - float((ref.f64(dx) * v.double()).sum())) < 40 * h * h + 80 * 2.0 ** -24 * 40 / h
        u = v[0] / v[0].norm()
        got = (f(x, w + h * u) - f(x, w - h * u)) / (2 * h)
        assert abs(got - float((ref.f64(dw) * u.double()).sum())) < 80 * 2.0 ** -24 * 40 / h


def test_norm_backward_of_nothing_and_repeats():
    dx, dw = mxq.mxq_rms_norm_backward(torch.zeros(0, 300, device=DEV), torch.zeros(0, 300, device=DEV), None, EPS,
                                       dweight=torch.full((300,), 7.0, device=DEV))
    assert dx.shape == (0, 300) and bool((dw == 0).all())
    g = gen(2)
    dy, x = (torch.randn(900, 520, generator=g).to(DEV) for _ in range(2))
    a, b = mxq.mxq_rms_norm_backward(dy, x, None, EPS), mxq.mxq_rms_norm_backward(dy, x, None, EPS)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_leading_dimensions_and_empty():
    x = torch.randn(3, 5, 200, generator=gen(1)).to(DEV)
    y, s = mxq.mxq_rms_norm(x, None, EPS, residual=x.float())
    assert y.shape == s.shape == x.shape
    flat, _ = mxq.mxq_rms_norm(x.view(15, 200), None, EPS, residual=x.float().view(15, 200))
    assert torch.equal(y.view(15, 200), flat)
    q, c, _, _ = mxq.mxq_rms_norm_fp8_group128(x[:0], None, EPS)
    assert q.shape == (0, 200) and c.shape == (0, 2)


def test_norm_operands_at_any_address():
    """Weights, rows and gradients that begin at odd elements; rows that all lie in one place are refused."""
    g = gen(9)
    buf = torch.randn(4000, generator=g)
    w = buf[3:3 + 264]
    x = values(40, 264, g, BF16)
    want, off = ref.norm(ref.f64(x), w, EPS)
    wd, xd = buf.to(DEV)[3:3 + 264], odd_view(x, 1, 3)
    y, _ = mxq.mxq_rms_norm(xd, wd, EPS)
    ref.check_values(y, want, off, "y")
    dy = values(40, 264, g, FP32, 2)
    (dx, dx_off), (dw, dw_off) = ref.norm_backward(dy, ref.f64(x), w, EPS, None)
    got, got_w = mxq.mxq_rms_norm_backward(odd_view(dy, 1, 1), xd, wd, EPS)
    ref.check_values(got, dx, dx_off, "dx")
    ref.check_values(got_w, dw, dw_off, "dweight")
    with pytest.raises(mxq.MxqError):
        mxq.mxq_rms_norm(x[:1].to(DEV).expand(5, 264), None, EPS)
    with pytest.raises(mxq.MxqError):
        mxq.mxq_rms_norm(x.to(DEV), None, 0.0)


def test_norm_leaves_the_rest_alone():
    """Outputs inside larger tensors: what lies around them keeps its values."""
    g = gen(6)
    x = torch.randn(6, 200, generator=g).to(DEV)
    y, s = torch.full((8, 210), 5.0, device=DEV), torch.full((8, 210), 5.0, device=DEV)
    q, c = torch.full((8, 210), 9, dtype=torch.uint8, device=DEV), torch.full((8, 4), 9, dtype=torch.uint8, device=DEV)
    mxq.mxq_rms_norm_fp8_group128(x, None, EPS, residual=x, residual_out=s[1:7, 3:203], y=y[1:7, 3:203], data=q[1:7, 3:203],
                                  scale=c[1:7, 1:3])
    for t, at, v in ((y, (slice(1, 7), slice(3, 203)), 5.0), (s, (slice(1, 7), slice(3, 203)), 5.0), (q, (slice(1, 7), slice(3, 203)), 9),
                     (c, (slice(1, 7), slice(1, 3)), 9)):
        keep = torch.ones_like(t, dtype=torch.bool)
        keep[at] = False
        assert bool((t[keep] == v).all())


def test_norm_captured_and_on_another_stream():
    g = gen(3)
    x, res, w = values(70, 1000, g, BF16).to(DEV), values(70, 1000, g, FP32).to(DEV), torch.randn(1000, generator=g).to(DEV)
    dy = values(70, 1000, g, BF16).to(DEV)

    def step(x, res, dy):
        q = mxq.mxq_rms_norm_fp8_group128_row_col(x, w, EPS, residual=res, with_y=True)
        return (*q, *mxq.mxq_rms_norm_backward(dy, q[4], w, EPS, dresidual=res))

    step(x, res, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step(x, res, dy)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, step(x, res, dy)))
    sx, sr, sd = x.clone(), res.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(sx, sr, sd)
    for k in range(4):
        sx.copy_(x.roll(k, 0) * (k + 1))
        sr.copy_(res.roll(k, 1))
        sd.copy_(dy * (0.5 + k))
        want = step(sx, sr, sd)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
