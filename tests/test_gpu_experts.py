"""Slots sorted by expert, rows brought into that order and back, and the gradients,
against plain forms."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check_sort(ids, n_experts):
    offsets, slots, position = mxq.mxq_sort_experts(ids.to(DEV), n_experts)
    want = ref.sort_experts(ids, n_experts)
    assert offsets.tolist() == want[0]
    assert slots.tolist() == want[1]
    assert position.shape == ids.shape and position.reshape(-1).tolist() == want[2]


@pytest.mark.parametrize("tokens,top_k,n", [(1, 1, 1), (1, 8, 8), (9, 6, 48), (63, 1, 2), (64, 3, 512), (300, 2, 5),
                                            (1024, 8, 33), (1025, 8, 64), (2048, 4, 7), (3000, 6, 160), (8193, 1, 511)])
def test_sort(tokens, top_k, n):
    g = gen(tokens + n)
    ids = torch.randint(0, n, (tokens, top_k), generator=g, dtype=torch.int32)
    check_sort(ids, n)
    dropped = torch.where(torch.rand(tokens, top_k, generator=g) < 0.2, torch.randint(-5, 0, (1,), generator=g).int(), ids)
    dropped[tokens // 2] = n                       # a token that no expert takes
    dropped[0, 0] = 2 ** 31 - 1
    check_sort(dropped, n)


@pytest.mark.parametrize("tokens", [5, 4000])
def test_sort_one_expert_takes_all_or_none(tokens):
    ids = torch.full((tokens, 4), 3, dtype=torch.int32)
    check_sort(ids, 9)
    check_sort(torch.full_like(ids, -1), 9)


def test_sort_of_a_strided_table_and_of_nothing():
    wide = torch.randint(-1, 6, (50, 10), generator=gen(1), dtype=torch.int32)
    want = ref.sort_experts(wide[:, 2:5], 6)
    offsets, slots, position = mxq.mxq_sort_experts(wide.to(DEV)[:, 2:5], 6)
    assert (offsets.tolist(), slots.tolist(), position.reshape(-1).tolist()) == want
    offsets, slots, position = mxq.mxq_sort_experts(torch.zeros((0, 4), dtype=torch.int32, device=DEV), 6)
    assert offsets.tolist() == [0] * 7 and slots.numel() == 0 and position.shape == (0, 4)


def routed(tokens, top_k, n, H, dtype, seed, drop=0.2):
    g = gen(seed)
    ids = torch.randint(0, n, (tokens, top_k), generator=g, dtype=torch.int32)
    ids = torch.where(torch.rand(tokens, top_k, generator=g) < drop, torch.tensor(-1, dtype=torch.int32), ids)
    ids[tokens // 2] = -1
    _, slots, position = ref.sort_experts(ids, n)
    w = torch.randn(tokens, top_k, generator=g)
    rows = torch.randn(tokens * top_k, H, generator=g).to(dtype)
    dy = torch.randn(tokens, H, generator=g).to(dtype)
    return slots, torch.tensor(position, dtype=torch.int32).view(tokens, top_k), w, rows, dy


CASES = [(1, 1, 1), (1, 6, 2048), (5, 2, 8), (33, 3, 100), (20, 8, 1001), (7, 9, 2056), (40, 4, 4096)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,top_k,H", CASES)
def test_dispatch_and_combine(tokens, top_k, H, dtype):
    slots, position, w, rows, dy = routed(tokens, top_k, 6, H, dtype, tokens + H)
    p64, w64, r64, g64 = position.long(), w.double(), rows.double(), dy.double()
    kept = p64 >= 0
    picked = torch.where(kept[..., None], r64[p64.clamp(min=0)], 0.0)
    half = torch.finfo(dtype).eps / 2
    # dropped rows hold NaN: they are not read
    for p in p64[~kept].reshape(-1).tolist():
        rows[~p] = float("nan")
    for odd in (False, True):
        def place(t):
            if not odd:
                return t.to(DEV)
            buf = torch.zeros((t.shape[0], t.shape[1] + 3), dtype=t.dtype, device=DEV)
            buf[:, 1:-2] = t.to(DEV)
            return buf[:, 1:-2]
        s, p = torch.tensor(slots, dtype=torch.int32, device=DEV), position.to(DEV)
        xs = mxq.mxq_dispatch_rows(place(dy), s, top_k)
        assert torch.equal(xs.cpu(), ref.gather(dy, slots, top_k))
        for weights, wv in ((w.to(DEV), w64), (None, torch.ones_like(w64))):
            y = mxq.mxq_combine_rows(place(rows), p, weights)
            terms = picked * wv[..., None]
            # one rounding of the sum, and 2 top_k fp32 roundings of products and partial sums
            allowed = half * terms.sum(1).abs() + 2 * top_k * 2.0 ** -24 * terms.abs().sum(1)
            assert bool(((y.cpu().double() - terms.sum(1)).abs() <= allowed * (1 + half)).all())
            drows, dw = mxq.mxq_combine_rows_backward(place(dy), place(rows), p, weights)
            want = torch.zeros_like(r64)
            want[p64[kept]] = (wv[..., None] * g64[:, None])[kept]
            assert bool(((drows.cpu().double() - want).abs() <= (half + 2.0 ** -24) * want.abs() * (1 + half)).all())
            prod = picked * g64[:, None]
            allowed = (H + 1) * 2.0 ** -24 * prod.abs().sum(-1)
            assert bool(((dw.cpu().double() - prod.sum(-1)).abs() <= allowed).all())
            assert (dw.cpu()[~kept] == 0).all()


def test_combine_ignores_positions_out_of_range():
    rows = torch.ones(4, 16, device=DEV)
    position = torch.tensor([[0, 4], [3, 2 ** 31 - 1], [-(2 ** 31), 1]], dtype=torch.int32, device=DEV)
    y = mxq.mxq_combine_rows(rows, position)
    assert torch.equal(y.cpu(), torch.ones(3, 16))
    drows = torch.full((4, 16), 5.0, device=DEV)
    drows, dw = mxq.mxq_combine_rows_backward(torch.ones(3, 16, device=DEV), rows, position, drows=drows)
    assert dw.tolist() == [[16, 0], [16, 0], [0, 16]]
    assert drows[:, 0].tolist() == [1, 1, 5, 1]          # no slot names row 2


def test_gradients_against_differences():
    """Small integers, so that sums and differences are exact."""
    tokens, top_k, H, g = 6, 3, 40, gen(2)
    slots, position, _, _, _ = routed(tokens, top_k, 4, H, torch.float32, 5)
    small = lambda *s: torch.randint(-3, 4, s, generator=g).float().to(DEV)
    rows, w, dy, p = small(tokens * top_k, H), small(tokens, top_k), small(tokens, H), position.to(DEV)
    f = lambda rows, w: float((mxq.mxq_combine_rows(rows, p, w) * dy).sum())
    drows, dw = mxq.mxq_combine_rows_backward(dy, rows, p, w)
    base = f(rows, w)
    for r in range(tokens * top_k):
        r2 = rows.clone()
        r2[r, r] += 1
        assert f(r2, w) - base == float(drows[r, r])
    for t in range(tokens):
        for j in range(top_k):
            w2 = w.clone()
            w2[t, j] += 1
            assert f(rows, w2) - base == float(dw[t, j])
    # the gradient of dispatch: combine without weights
    x, s = small(tokens, H), torch.tensor(slots, dtype=torch.int32, device=DEV)
    seed = small(tokens * top_k, H)
    dx = mxq.mxq_combine_rows(seed, p)
    h = lambda x: float((mxq.mxq_dispatch_rows(x, s, top_k) * seed).sum())
    for t in range(tokens):
        x2 = x.clone()
        x2[t, t] += 1
        assert h(x2) - h(x) == float(dx[t, t])


def test_routing_repeats_on_streams_and_in_graphs():
    tokens, top_k, n, H = 1500, 6, 40, 256
    ids = torch.randint(-1, n, (tokens, top_k), generator=gen(3), dtype=torch.int32).to(DEV)
    x, w = torch.randn(tokens, H, device=DEV).to(torch.bfloat16), torch.rand(tokens, top_k, device=DEV)

    def step():
        offsets, slots, position = mxq.mxq_sort_experts(ids, n)
        xs = mxq.mxq_dispatch_rows(x, slots, top_k)
        y = mxq.mxq_combine_rows(xs, position, w)
        return (offsets, slots, position, xs, y) + mxq.mxq_combine_rows_backward(y, xs, position, w)

    def same(got, want):
        for a, b in zip(got, want):
            assert torch.equal(a, b)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        ids.copy_(torch.randint(-1, n, (tokens, top_k), generator=gen(50 + k), dtype=torch.int32).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        same(out, step())
