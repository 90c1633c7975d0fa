"""Every kernel of the FP8 products against plain 64-bit forms, at sizes chosen from the
library's rule (tests/product_sizes.py), with ragged edges and ragged experts."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import fp8_ref as ref
from tests.product_sizes import CASES, offsets_of
from tests.test_gpu_products import DEV, check_fast, codes, dev, gen, payload

pytestmark = pytest.mark.gpu


def odd(t):
    """The same values on the device at an odd address with odd row and matrix strides."""
    rows, cols = t.shape[-2:]
    ld, n = cols + 5 - cols % 2, t.shape[0] if t.dim() == 3 else 1
    step = rows * ld + 3
    buf = torch.zeros(3 + n * step, dtype=t.dtype, device=DEV)
    v = buf.as_strided((n, rows, cols), (step, ld, 1), 3)
    v.copy_(t.reshape(n, rows, cols))
    return v if t.dim() == 3 else v[0]


def operands(c, g, code=codes):
    """The case's operands on the host: V with its codes, U with its codes, and the rows' offsets."""
    ceil = ref.ceil_div
    lead = (c.experts,) if c.experts else ()
    if c.mode == "dw":
        groups = c.R // 128 + c.experts if c.experts else ceil(c.R)
        return payload(g, c.R, c.I), code(g, groups, c.I), payload(g, c.R, c.J), code(g, groups, c.J), offsets_of(c.R, c.experts)
    n, k = (c.J, c.R) if c.mode == "y" else (c.R, c.J)
    return (payload(g, c.I, c.R), code(g, c.I, ceil(c.R)), payload(g, *lead, n, k), code(g, *lead, ceil(n), ceil(k)),
            offsets_of(c.I, c.experts))


def call(c, place, v, vc, u, uc, offsets, **kw):
    kw["offsets"] = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    if c.mode == "dw":
        return mxq.mxq_matmul_fp8_group128_wgrad(place(v), place(vc), place(u), place(uc), **kw)
    fn = mxq.mxq_matmul_fp8_block128 if c.mode == "y" else mxq.mxq_matmul_fp8_block128_dgrad
    return fn(place(v), place(vc), place(u), place(uc), fast_accum=c.fast, **kw)


def expected(c, v, vc, u, uc, offsets):
    if c.mode == "dw":
        return ref.wgrad(v, vc, u, uc, offsets)
    return ref.matmul(v, vc, u, uc, offsets, transpose=c.mode == "dx")


@pytest.mark.parametrize("c", CASES, ids=str)
def test_kernel(c):
    a = operands(c, gen(c.I + 3 * c.R + 7 * c.J + c.experts))
    want = expected(c, *a)
    check = check_fast if c.fast else ref.check
    for dtype in (torch.float32, torch.bfloat16):
        out = call(c, dev if c.fed else odd, *a, out_dtype=dtype)
        check(out, *want, c.R, f"{c} {dtype}")


SPECIAL = [c for c in CASES if c.kernel.startswith("kExact")]


@pytest.mark.parametrize("c", SPECIAL, ids=str)
def test_codes_of_every_kind_in_one_reduction(c):
    """Sums in fp32 where some blocks' codes cannot go into the conversion to bf16: codes far from 127, 0
    among them, NaN codes and payloads, in some rows and columns of some blocks."""
    g = gen(c.I + c.R + c.J)

    def kinds(g, *shape):
        t = codes(g, *shape)
        pick = torch.rand(shape, generator=g)
        t = torch.where(pick < 0.02, torch.tensor(0, dtype=torch.uint8), t)
        t = torch.where((pick >= 0.02) & (pick < 0.03), torch.tensor(60, dtype=torch.uint8), t)
        return torch.where((pick >= 0.03) & (pick < 0.04), torch.tensor(169, dtype=torch.uint8), t)

    v, vc, u, uc, offsets = operands(c, g, kinds)
    vc[0, 0], uc[..., 0, 0] = 0, 60
    blocks = vc if c.mode == "dw" else vc.t()            # [reduction block, row]
    blocks[0, 5], blocks[-1, 7] = 175, 255
    v[-1 if c.mode == "dw" else 3, 11], u[..., 17, 9] = 0x7F, 0xFF
    want = expected(c, v, vc, u, uc, offsets)
    assert 0 < int(torch.isnan(want[0]).sum()) < want[0].numel() // 2
    out = call(c, dev if c.fed else odd, v, vc, u, uc, offsets, out_dtype=torch.float32)
    ref.check(out, *want, c.R, str(c))


@pytest.mark.parametrize("c", SPECIAL, ids=str)
@pytest.mark.parametrize("pair", [(0, 0), (0, 254), (254, 0), (1, 127), (76, 127), (127, 168), (77, 77), (167, 167), (168, 60)])
def test_one_code_for_all(c, pair):
    """The lowest and highest codes, and those beside the borders of the two ways to sum."""
    v, vc, u, uc, offsets = operands(c, gen(c.I * c.J + pair[0]))
    vc.fill_(pair[0]), uc.fill_(pair[1])
    out = call(c, dev if c.fed else odd, v, vc, u, uc, offsets, out_dtype=torch.float32)
    ref.check(out, *expected(c, v, vc, u, uc, offsets), c.R, f"{c} {pair}")
