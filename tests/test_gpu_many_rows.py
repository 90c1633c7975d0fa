"""Row counts that need more lanes than one launch has (2^32 in a dimension), against torch."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def bf16(g, *shape):
    """Small integers: their products and short sums are exact."""
    return torch.randint(-4, 5, shape, generator=g, device=DEV, dtype=torch.int16).to(torch.bfloat16)


def test_combine_gradients_of_many_tokens():
    """256 lanes a token."""
    tokens, H, g = (1 << 24) + 3, 8, gen(1)
    dy, rows = bf16(g, tokens, H), bf16(g, tokens, H)
    position = torch.randperm(tokens, generator=g, device=DEV).int().view(tokens, 1)
    position[5] = ~position[5]
    w = torch.randint(1, 4, (tokens, 1), generator=g, device=DEV).float()
    drows, dw = mxq.mxq_combine_rows_backward(dy, rows, position, w)
    kept = (position >= 0).float()
    at = torch.where(position >= 0, position, ~position).view(-1).long()
    assert torch.equal(drows[at].float(), dy.float() * w * kept)
    assert torch.equal(dw, (dy.float() * rows[at].float()).sum(1, keepdim=True) * kept)


@pytest.mark.parametrize("gathered", [False, True])
def test_quantize_rows_of_many_groups(gathered):
    """16 lanes a group.  Values on the E4M3 grid: each group's code is its one value's own."""
    rows, g = (1 << 28) + 9, gen(2)
    x = torch.randint(0, 127, (rows, 1), generator=g, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn)
    x = x.to(torch.bfloat16)
    slots = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device=DEV) if gathered else None
    q, codes = mxq.mxq_quantize_fp8_group128(x, slots=slots)
    if gathered:
        x = x.flip(0)
    for lo in range(0, rows, 1 << 26):           # a part at a time: the values in 64 bits are 8 bytes each
        part = slice(lo, min(rows, lo + (1 << 26)))
        value = q[part].view(torch.float8_e4m3fn).double() * torch.exp2(codes[part].double() - 127)
        assert torch.equal(value, x[part].double())
        assert bool(((codes[part] == 0) == (x[part] == 0)).all())


@pytest.mark.parametrize("experts", [0, 3])
def test_quantize_columns_of_many_rows(experts):
    """More than 65535 tiles of 128 rows, by expert or not."""
    rows, K, g = 65536 * 128 * 2 + 300, 3, gen(3)
    x = torch.randint(0, 127, (rows, K), generator=g, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn)
    x = x.to(torch.bfloat16)
    ends = [0, 77, rows // 2 + 1, rows - 5] if experts else [0, rows]
    offsets = torch.tensor(ends, dtype=torch.int32, device=DEV) if experts else None
    rq, rc, q, codes = mxq.mxq_quantize_fp8_group128_row_col(x, offsets=offsets)
    q2, codes2 = mxq.mxq_quantize_fp8_group128_col(x, offsets=offsets)
    assert torch.equal(q, q2) and torch.equal(codes, codes2)
    one = mxq.mxq_quantize_fp8_group128(x)
    assert torch.equal(rq, one[0]) and torch.equal(rc, one[1])
    first = 0
    for lo, hi in zip(ends, ends[1:]):           # each expert's groups, transposed, are a row's
        n = (hi - lo + 127) // 128
        part = torch.zeros((n * 128, K), dtype=x.dtype, device=DEV)
        part[:hi - lo] = x[lo:hi]
        groups = part.view(n, 128, K).transpose(1, 2).reshape(n * K, 128).contiguous()
        wq, wc = mxq.mxq_quantize_fp8_group128(groups)
        assert torch.equal(codes[first:first + n], wc.view(n, K))
        assert torch.equal(q[lo:hi], wq.view(n, K, 128).transpose(1, 2).reshape(n * 128, K)[:hi - lo])
        first += n
    assert (codes[first:] == 0).all() and (q[ends[-1]:] == 0).all()


def test_many_wide_rows_into_order_and_back():
    """More than 2^34 elements of the result, at 8 a lane."""
    rows, H, few, g = (1 << 21) + 3, 8192, 1000, gen(4)
    x, at = bf16(g, few, H), torch.randint(0, few, (rows,), generator=g, device=DEV, dtype=torch.int32)
    at[17] = -1
    for name in ("dispatch", "combine"):
        out = mxq.mxq_dispatch_rows(x, at, 1) if name == "dispatch" else mxq.mxq_combine_rows(x, at.view(rows, 1))
        assert (out[17] == 0).all()
        for lo in range(0, rows, 1 << 17):
            part = slice(lo, min(rows, lo + (1 << 17)))
            want = x[at[part].clamp(min=0).long()]
            want[at[part] < 0] = 0
            assert torch.equal(out[part], want), f"{name}, rows from {lo}"
        del out


def e4m3(g, *shape):
    """Small integers in E4M3."""
    return torch.randint(-4, 5, shape, generator=g, device=DEV, dtype=torch.int16).to(torch.float32).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("fast", [False, True])
def test_products_of_many_rows(fast):
    """More than 65535 tiles of 128 rows that begin at odd addresses."""
    M, N, K, g = 65536 * 128 + 5, 70, 17, gen(5)
    x, w = e4m3(g, M, K), e4m3(g, N, K)
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=DEV)
    y = mxq.mxq_matmul_fp8_block128(x, one(M, 1), w, one(1, 1), out_dtype=torch.float32, fast_accum=fast)
    assert torch.equal(y, x.float() @ w.float().t())
    dx = mxq.mxq_matmul_fp8_block128_dgrad(x, one(M, 1), w.t().contiguous(), one(1, 1), out_dtype=torch.float32,
                                           fast_accum=fast)
    assert torch.equal(dx, y)


@pytest.mark.parametrize("fast", [False, True])
def test_products_of_many_columns(fast):
    """2^29 columns and more, at 8 lanes a column."""
    J, g = (1 << 29) + 200, gen(6)
    x, w = e4m3(g, 1, 1), e4m3(g, J, 1)
    x[0, 0] = 3
    tiles = torch.randint(120, 131, ((J + 127) // 128, 1), generator=g, device=DEV, dtype=torch.uint8)
    one = torch.full((1, 1), 127, dtype=torch.uint8, device=DEV)
    y = mxq.mxq_matmul_fp8_block128(x, one, w, tiles, fast_accum=fast)
    dx = mxq.mxq_matmul_fp8_block128_dgrad(x, one, w.t(), tiles.t(), fast_accum=fast)
    for lo in range(0, J, 1 << 26):
        part = slice(lo, min(J, lo + (1 << 26)))
        scale = torch.exp2(tiles[lo // 128:(part.stop + 127) // 128].float() - 127).repeat_interleave(128)[:part.stop - lo]
        want = (3 * w[part, 0].float() * scale).bfloat16()
        assert torch.equal(y[0, part], want) and torch.equal(dx[0, part], want), f"columns from {lo}"
    if not fast:
        codes = torch.randint(120, 131, (1, J), generator=g, device=DEV, dtype=torch.uint8)
        dw = mxq.mxq_matmul_fp8_group128_wgrad(x, one, w.t(), codes, out_dtype=torch.bfloat16)
        for lo in range(0, J, 1 << 26):
            part = slice(lo, min(J, lo + (1 << 26)))
            want = (3 * w[part, 0].float() * torch.exp2(codes[0, part].float() - 127)).bfloat16()
            assert torch.equal(dw[0, part], want), f"columns from {lo}"
