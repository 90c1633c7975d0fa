"""Refusals of the FP8 quantizer, products and expert routing, on the host: every
bad argument is found before anything is enqueued (fake addresses; no GPU is
touched), and the plain forms that the GPU tests use hold what they claim."""
import ctypes

import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from microscaling_weight_quantization_amd import build as B
from tests import fp8_ref as ref

OK, NULL, SHAPE, DTYPE, ALIAS = mxq.MXQ_OK, mxq.MXQ_ERR_NULL, mxq.MXQ_ERR_SHAPE, mxq.MXQ_ERR_DTYPE, mxq.MXQ_ERR_ALIAS
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    if B.stale():
        B.build(["libmxq.so"])
    return mxq.load()


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults), set(kw) - set(defaults)
    return fn(*{**defaults, **kw}.values())


# 200 rows of 300: bf16 120000 bytes, payload 60000, row codes 200 x 3, column codes 2 x 300
QUANT = dict(x=0x100000, ld_x=300, x_rows=200, rows=200, K=300, dt=0, slots=None, top_k=1)


def refused_like_quantize(fn, d, narrow):
    assert call(fn, d, dt=mxq.MXQ_FP16) == DTYPE
    assert call(fn, d, dt=9) == DTYPE
    assert call(fn, d, x=None) == NULL
    for k in ("rows", "K", "x_rows"):
        assert call(fn, d, **{k: -1}) == SHAPE
        assert call(fn, d, **{k: (1 << 30) + 1}) == SHAPE
    assert call(fn, d, rows=201) == SHAPE                         # more rows than x has
    assert call(fn, d, slots=0x900000, top_k=0) == SHAPE
    assert call(fn, d, slots=0x900002, top_k=1) == SHAPE          # not an int32 address
    assert call(fn, d, x=0x100001) == SHAPE                       # not a bf16 address
    assert call(fn, d, ld_x=299) == SHAPE
    assert call(fn, d, ld_x=BIG) == SHAPE
    for k, v in narrow.items():
        assert call(fn, d, **{k: v}) == SHAPE, k
        assert call(fn, d, **{k: BIG}) == SHAPE, k
    for k in [k for k in d if k.endswith(("data", "scale")) and not k.startswith("ld")]:
        assert call(fn, d, **{k: None}) == NULL, k
        assert call(fn, d, **{k: 0x100000 + 119999}) == ALIAS, k  # the last byte of x
        assert call(fn, d, slots=0x900000, **{k: 0x900000 + 799}) == ALIAS, k
    assert call(fn, d, rows=0) == OK                              # empty: nothing is enqueued
    assert call(fn, d, K=0, x=None) == OK


def test_quantize_refusals(lib):
    d = dict(QUANT, data=0x200000, ld_data=300, scale=0x300000, scale_ld=3, stream=None)
    refused_like_quantize(lib.mxq_quantize_fp8_group128, d, {"ld_data": 299, "scale_ld": 2})
    assert call(lib.mxq_quantize_fp8_group128, d, scale=0x200000 + 59999) == ALIAS
    assert call(lib.mxq_quantize_fp8_group128, d, scale_ld=2) == SHAPE


def test_quantize_columns_refusals(lib):
    d = dict(QUANT, offsets=None, n=0, data=0x200000, ld_data=300, scale=0x300000, scale_ld=300, stream=None)
    fn = lib.mxq_quantize_fp8_group128_col
    refused_like_quantize(fn, d, {"ld_data": 299, "scale_ld": 299})
    assert call(fn, d, scale=0x200000 + 59999) == ALIAS
    for n in (0, -1, 513):
        assert call(fn, d, offsets=0x800000, n=n) == SHAPE
    assert call(fn, d, offsets=0x800001, n=4) == SHAPE
    assert call(fn, d, offsets=0x200000, n=4) == ALIAS
    # with 4 experts there are 1 + 4 code rows
    assert call(fn, d, offsets=0x300000 + 4 * 300, n=4) == ALIAS
    both = dict(QUANT, offsets=None, n=0, row_data=0x200000, ld_row=300, row_scale=0x300000, row_scale_ld=3,
                col_data=0x400000, ld_col=300, col_scale=0x500000, col_scale_ld=300, stream=None)
    fn = lib.mxq_quantize_fp8_group128_row_col
    refused_like_quantize(fn, both, {"ld_row": 299, "row_scale_ld": 2, "ld_col": 299, "col_scale_ld": 299})
    assert call(fn, both, col_data=0x200000 + 59999) == ALIAS
    assert call(fn, both, col_scale=0x300000 + 599) == ALIAS


# 200 x 300 times 260 x 300: y 200 x 260, bf16
PRODUCT = dict(v=0x100000, ld_v=300, v_scale=0x200000, v_scale_ld=3, w=0x300000, ld_w=300, w_stride=0, tiles=0x400000,
               tile_ld=3, tile_stride=0, M=200, N=260, K=300, offsets=None, n=0, out=0x500000, ld_out=260, dt=0,
               fast=0, stream=None)


@pytest.mark.parametrize("which", ["y", "dx"])
def test_product_refusals(lib, which):
    fn = lib.mxq_matmul_fp8_block128 if which == "y" else lib.mxq_matmul_fp8_block128_dgrad
    d = dict(PRODUCT) if which == "y" else dict(PRODUCT, ld_v=260, ld_out=300)
    assert call(fn, d, dt=mxq.MXQ_FP16) == DTYPE
    for k in ("v", "v_scale", "w", "tiles", "out"):
        assert call(fn, d, **{k: None}) == NULL, k
    for k in ("M", "N", "K"):
        assert call(fn, d, **{k: -1}) == SHAPE
        assert call(fn, d, **{k: (1 << 30) + 1}) == SHAPE
    for k in ("ld_v", "v_scale_ld", "ld_w", "tile_ld", "ld_out"):
        assert call(fn, d, **{k: d[k] - 1}) == SHAPE, k
        assert call(fn, d, **{k: BIG}) == SHAPE, k
    assert call(fn, d, out=0x500001) == SHAPE
    for k in ("v", "v_scale", "w", "tiles"):
        assert call(fn, d, out=d[k]) == ALIAS, k
    # experts: as many weights, so far apart
    e = dict(d, offsets=0x800000, n=3, w_stride=260 * 300, tile_stride=9)
    assert call(fn, e, n=0) == SHAPE and call(fn, e, n=513) == SHAPE
    assert call(fn, e, offsets=0x800002) == SHAPE
    assert call(fn, e, w_stride=260 * 300 - 1) == SHAPE
    assert call(fn, e, tile_stride=8) == SHAPE
    assert call(fn, e, w_stride=BIG) == SHAPE
    assert call(fn, e, out=0x300000 + 2 * 260 * 300) == ALIAS     # the last expert's weight
    assert call(fn, e, out=0x800000) == ALIAS
    # empty outputs
    assert call(fn, d, M=0, out=None, v=None, v_scale=None) == OK


def test_weight_gradient_refusals(lib):
    fn = lib.mxq_matmul_fp8_group128_wgrad
    d = dict(dy=0x100000, ld_dy=260, dy_scale=0x200000, dy_scale_ld=260, x=0x300000, ld_x=300, x_scale=0x400000,
             x_scale_ld=300, M=200, N=260, K=300, offsets=None, n=0, dw=0x600000, ld_dw=300, dw_stride=0, dt=1,
             stream=None)
    assert call(fn, d, dt=5) == DTYPE
    for k in ("dy", "dy_scale", "x", "x_scale", "dw"):
        assert call(fn, d, **{k: None}) == NULL, k
    for k in ("ld_dy", "dy_scale_ld", "ld_x", "x_scale_ld", "ld_dw"):
        assert call(fn, d, **{k: d[k] - 1}) == SHAPE, k
        assert call(fn, d, **{k: BIG}) == SHAPE, k
    for k in ("dy", "dy_scale", "x", "x_scale"):
        assert call(fn, d, dw=d[k]) == ALIAS, k
    e = dict(d, offsets=0x900000, n=3, dw_stride=260 * 300)
    assert call(fn, e, dw_stride=260 * 300 - 1) == SHAPE
    assert call(fn, e, dw=0x900000 - 3 * 260 * 300 * 4 + 4) == ALIAS   # the last gradient over the offsets
    assert call(fn, e, n=513) == SHAPE
    assert call(fn, d, N=0, dw=None) == OK and call(fn, d, K=0) == OK


def test_sort_refusals(lib):
    fn = lib.mxq_sort_experts
    d = dict(ids=0x100000, ld=6, T=9, k=6, n=48, offsets=0x200000, slots=0x300000, position=0x400000, ws=None, bytes=0,
             stream=None)
    for k in ("ids", "offsets", "slots", "position"):
        assert call(fn, d, **{k: None}) == NULL, k
        assert call(fn, d, **{k: d[k] + 2}) == SHAPE, k
    assert call(fn, d, ld=5) == SHAPE and call(fn, d, T=-1) == SHAPE and call(fn, d, k=0) == SHAPE
    assert call(fn, d, n=0) == SHAPE and call(fn, d, n=513) == SHAPE
    assert call(fn, d, T=1 << 30, k=2, ld=2) == SHAPE
    for k in ("offsets", "slots", "position"):
        assert call(fn, d, **{k: 0x100000 + 4 * 53}) == ALIAS, k
    assert call(fn, d, position=0x300000 + 4 * 53) == ALIAS
    # a large table needs its workspace
    need = lib.mxq_sort_experts_workspace(4096, 6, 48)
    assert need > 0 and need % 4 == 0
    assert lib.mxq_sort_experts_workspace(9, 6, 48) == 0
    assert lib.mxq_sort_experts_workspace(-1, 6, 48) == 0
    big = dict(d, T=4096, ws=0x800000, bytes=need)
    assert call(fn, big, ws=None) == NULL
    assert call(fn, big, bytes=need - 1) == SHAPE
    assert call(fn, big, ws=0x800001) == SHAPE
    assert call(fn, big, ws=0x400000 + 4 * 4096 * 6 - 4) == ALIAS


def test_row_movers_refusals(lib):
    d = dict(x=0x100000, ld_x=64, x_rows=10, slots=0x200000, rows=30, k=3, H=64, dt=0, out=0x300000, ld_out=64,
             stream=None)
    fn = lib.mxq_dispatch_rows
    assert call(fn, d, dt=2) == DTYPE
    for k in ("x", "slots", "out"):
        assert call(fn, d, **{k: None}) == NULL, k
    for k in ("ld_x", "ld_out"):
        assert call(fn, d, **{k: 63}) == SHAPE and call(fn, d, **{k: BIG}) == SHAPE
    assert call(fn, d, k=0) == SHAPE and call(fn, d, rows=-1) == SHAPE and call(fn, d, x_rows=-1) == SHAPE
    assert call(fn, d, slots=0x200001) == SHAPE and call(fn, d, out=0x300001) == SHAPE
    assert call(fn, d, out=0x100000 + 10 * 128 - 2) == ALIAS and call(fn, d, out=0x200000) == ALIAS
    assert call(fn, d, rows=0, out=None) == OK and call(fn, d, H=0) == OK

    d = dict(rows=0x100000, ld_rows=64, n_rows=30, position=0x200000, weights=0x280000, T=10, k=3, H=64, dt=1,
             y=0x300000, ld_y=64, stream=None)
    fn = lib.mxq_combine_rows
    assert call(fn, d, dt=2) == DTYPE
    for k in ("rows", "position", "y"):
        assert call(fn, d, **{k: None}) == NULL, k
    for k in ("ld_rows", "ld_y"):
        assert call(fn, d, **{k: 63}) == SHAPE and call(fn, d, **{k: BIG}) == SHAPE
    assert call(fn, d, T=1 << 29) == SHAPE                        # slots past 2^30
    for k in ("rows", "position", "weights"):
        assert call(fn, d, y=d[k]) == ALIAS, k
    assert call(fn, d, T=0, y=None) == OK

    d = dict(dy=0x100000, ld_dy=64, rows=0x180000, ld_rows=64, n_rows=30, position=0x200000, weights=0x280000, T=10,
             k=3, H=64, dt=1, drows=0x300000, ld_drows=64, dw=0x380000, stream=None)
    fn = lib.mxq_combine_rows_backward
    assert call(fn, d, dt=2) == DTYPE
    for k in ("dy", "rows", "position", "drows"):
        assert call(fn, d, **{k: None}) == NULL, k
    for k in ("ld_dy", "ld_rows", "ld_drows"):
        assert call(fn, d, **{k: 63}) == SHAPE, k
    for k in ("dy", "rows", "position", "weights", "drows"):
        assert call(fn, d, dw=d[k]) == ALIAS, k
    assert call(fn, d, drows=0x100000) == ALIAS and call(fn, d, dw=0x380001) == SHAPE
    assert call(fn, d, T=0) == OK


def test_binding_checks_extents():
    """Shapes that do not belong together raise ValueError before the library is called."""
    b = lambda *s: torch.zeros(s, dtype=torch.uint8)
    with pytest.raises(ValueError, match="tile_code"):
        mxq._weights(b(200, 300), b(2, 2), 0)
    with pytest.raises(ValueError, match="n_experts"):
        mxq._weights(b(200, 300), b(2, 3), 4)
    with pytest.raises(ValueError, match="n_experts"):
        mxq._weights(b(3, 200, 300), b(3, 2, 3), 4)
    with pytest.raises(ValueError, match="bytes"):
        mxq._weights(torch.zeros(200, 300), b(2, 3), 0)
    with pytest.raises(ValueError, match="contiguous"):
        mxq._weights(b(300, 200).t(), b(2, 3), 0)
    assert mxq._weights(b(4, 200, 300), b(4, 2, 3), 4)[:2] == (200, 300)
    with pytest.raises(ValueError, match="holds bytes"):
        mxq._rows_operand(b(5, 299), b(5, 3), 300, "x")
    with pytest.raises(ValueError, match="must cover"):
        mxq._rows_operand(b(5, 300), b(5, 2), 300, "x")
    with pytest.raises(ValueError, match="must cover"):
        mxq._rows_operand(b(5, 300), b(4, 3), 300, "x")
    with pytest.raises(ValueError, match="int32"):
        mxq._experts_of(torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="n_experts"):
        mxq._experts_of(torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="elements"):
        mxq._slots_of(torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="output"):
        mxq._result(b(1), torch.zeros(3, 4), (3, 5), torch.float32)


def test_binding_refuses_host_tensors():
    f, b, i = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.int32)
    calls = [lambda: mxq.mxq_quantize_fp8_group128(f), lambda: mxq.mxq_quantize_fp8_group128_col(f),
             lambda: mxq.mxq_quantize_fp8_group128_row_col(f), lambda: mxq.mxq_matmul_fp8_block128(b, b, b, b),
             lambda: mxq.mxq_matmul_fp8_block128_dgrad(b, b, b, b),
             lambda: mxq.mxq_matmul_fp8_group128_wgrad(b, b, b, b), lambda: mxq.mxq_sort_experts(i, 4),
             lambda: mxq.mxq_dispatch_rows(f, i.view(-1), 2), lambda: mxq.mxq_combine_rows(f, i),
             lambda: mxq.mxq_combine_rows_backward(f, f, i)]
    for c in calls:
        with pytest.raises(ValueError, match="device tensors"):
            c()


# ---- the plain forms ---------------------------------------------------------------------

def test_plain_quantizer_against_its_definition():
    """Every value is the nearest of the grid at the smallest scale that does not saturate."""
    g = torch.Generator().manual_seed(1)
    grid = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double()
    grid = grid[torch.isfinite(grid)]
    for k in (-140, -120, 0, 100):
        v = torch.randn(128, generator=g, dtype=torch.float64).to(torch.float32).double() * 2.0 ** k
        q, code = ref.quantize_group(v)
        s = 2.0 ** (code - 127)
        amax = float(v.abs().max())
        assert amax <= 448 * s and (code == 0 or amax > 448 * s / 2)
        off = (ref.payload_values(q) - v / s).abs()
        assert torch.equal(off, (grid[None] - (v / s)[:, None]).abs().min(1).values)


def test_plain_segments_and_sort():
    assert ref.segments([0, 250, 100, 5000, -3, 280], 300) == [(0, 250), (250, 250), (250, 300), (300, 300), (300, 300)]
    assert ref.segments(None, 7) == [(0, 7)]
    ids = torch.tensor([[1, 0], [9, 1], [0, -1]])
    assert ref.sort_experts(ids, 2) == ([0, 2, 4], [1, 4, 0, 3, ~2, ~5], [2, 0, ~4, 3, 1, ~5])
