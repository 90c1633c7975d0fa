"""Refusals of calls by expert on no rows, on the host (fake addresses; nothing is enqueued): the code rows are written, so
their place is checked; without one, or without columns, there is nothing to do."""
import pytest

import microscaling_weight_quantization_amd as mxq
from microscaling_weight_quantization_amd import build as B

OK, SHAPE, ALIAS = mxq.MXQ_OK, mxq.MXQ_ERR_SHAPE, mxq.MXQ_ERR_ALIAS


@pytest.fixture(scope="module")
def lib():
    if B.stale():
        B.build(["libmxq.so"])
    return mxq.load()


CODES = dict(offsets=0x100000, n=4)
QUANT = dict(x=None, ld_x=300, x_rows=0, rows=0, K=300, dt=0, slots=None, top_k=1, **CODES)
ROW = dict(data=None, ld=300, scale=None, scale_ld=3)
COL = dict(cdata=None, ld_col=300, cscale=0x200000, cscale_ld=300, stream=None)


@pytest.mark.parametrize("name,d", [
    ("mxq_quantize_fp8_group128_col", dict(QUANT, **COL)),
    ("mxq_quantize_fp8_group128_row_col", dict(QUANT, **ROW, **COL)),
    ("mxq_activate_fp8_group128_row_col", dict(gate=None, ld_gate=300, up=None, ld_up=300, rows=0, K=300, dt=0, act=0, **CODES, **ROW, **COL)),
    ("mxq_activate_fp8_group128_backward", dict(da=None, ld_da=300, gate=None, ld_gate=300, up=None, ld_up=300, rows=0, K=300, dt=0, act=0,
                                                **CODES, **ROW, **COL)),
])
def test_no_rows_refusals(lib, name, d):
    call = lambda **kw: getattr(lib, name)(*{**d, **kw}.values())
    assert call(cscale_ld=299) == SHAPE and call(cscale_ld=1 << 62) == SHAPE and call(offsets=0x100002) == SHAPE
    assert call(n=0) == SHAPE and call(n=513) == SHAPE
    assert call(cscale=0x100000 + 19) == ALIAS and call(offsets=0x200000 + 3 * 300 + 296) == ALIAS
    assert call(cscale=None, cscale_ld=0) == OK and call(K=0) == OK and call(offsets=None, n=0) == OK
    if name.endswith("backward"):   # both halves' codes
        assert call(up=0x300000) == SHAPE and call(up=0x300000, cscale_ld=600, offsets=0x200000 + 4 * 600 - 4) == ALIAS
