"""Tokens to experts and the gradient of the router's logits against the definition in 64
bits: every size of choice, groups, biases, ties, closed experts, masked tokens, values that are not finite,
scores next to each other, strides, captured."""
import math

import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import between_ref as ref
from tests.test_gpu_products import odd_view

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
INF = float("inf")
# a score in fp32: the exponential and what stands in it (logits of up to 16 in these tests, a half step of each), the sum, the quotients
REL = 2 * (16 + 24) * ref.HALF


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check(logits, top_k, place=lambda t: t.to(DEV), **how):
    ids, w = mxq.mxq_route_experts(place(logits), top_k, **{k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in how.items()})
    want, want_w = ref.route(logits, top_k, **how)
    assert ids.dtype == torch.int32 and torch.equal(ref.host(ids), want), "ids"
    ref.check_values(w, want_w, want_w.abs() * REL, "weights")
    back = {k: how[k] for k in ("score", "renormalize", "scale") if k in how}
    dw = torch.randn(want_w.shape, generator=gen(top_k))
    got = mxq.mxq_route_experts_backward(dw.to(DEV), place(logits), ids, **back)
    grad, size = ref.route_backward(dw, logits, want, **back)
    assert got.dtype == logits.dtype
    ref.check_values(got, grad, size * 2 * REL, "dlogits")


def logits_of(T, E, seed, dtype=FP32, spread=1.5):
    return (spread * torch.randn(T, E, generator=gen(seed))).to(dtype)


SIZES = [(1, 1, 1), (1, 4, 1), (9, 48, 6), (5, 64, 8), (7, 65, 3), (33, 128, 8), (3, 160, 6), (17, 256, 8), (4, 511, 10), (6, 512, 1), (2, 512, 512),
         (2, 300, 70), (130, 7, 7)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route_sizes(T, E, k, score, dtype):
    l = logits_of(T, E, T + E, dtype)
    check(l, k, score=score)
    check(l, k, score=score, renormalize=False, scale=2.5)
    check(l, k, odd_view, score=score, bias=0.2 * torch.randn(E, generator=gen(E)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (160, 8, 3, 6), (48, 6, 1, 8), (64, 64, 9, 9), (96, 3, 3, 5), (12, 4, 2, 6), (512, 256, 5, 9)])
def test_route_groups(E, groups, top, k, score):
    for group_top in (1, 2):
        for bias in (None, 0.1 * torch.randn(E, generator=gen(E))):
            for dtype in (BF16, FP32):
                check(logits_of(19, E, E + top, dtype), k, score=score, n_groups=groups, top_groups=top, group_top=group_top, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties(score):
    """Equal logits, equal biased scores and equal groups: the lower index."""
    l = torch.randint(-2, 3, (40, 96), generator=gen(1)).float()
    for how in ({}, {"bias": torch.zeros(96)}, {"n_groups": 8, "top_groups": 3}, {"n_groups": 8, "top_groups": 3, "group_top": 2},
                {"bias": torch.randint(0, 2, (96,), generator=gen(2)).float(), "n_groups": 4, "top_groups": 2, "group_top": 2}):
        check(l, 6, score=score, **how)
    check(torch.zeros(3, 200), 9, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_closed_experts_and_masked_tokens(score):
    l = logits_of(50, 64, 4)
    l[:, 5:40] = -INF
    l[7] = -INF
    l[8, :] = -INF
    l[8, 33] = 0.5
    l[9, 40:] = -INF
    mask = torch.rand(50, generator=gen(5)) < 0.7
    bias = 0.1 * torch.randn(64, generator=gen(6))
    closed = bias.clone()
    closed[50:60] = -INF
    for b in (None, bias, closed):
        for how in ({}, {"n_groups": 8, "top_groups": 3, "group_top": 2}, {"n_groups": 8, "top_groups": 8}):
            check(l, 8, score=score, bias=b, **how)
            check(l, 8, score=score, bias=b, mask=mask, renormalize=False, **how)
    check(l, 8, score=score, mask=torch.zeros(50, dtype=torch.bool))
    check(l, 8, score=score, mask=mask.to(torch.uint8) * 7)


def test_route_far_apart():
    """Scores that underflow still make weights that sum to 1, and small gradients stay what they are."""
    l = torch.tensor([[0.0, -200.0, -201.0, -400.0], [90.0, 0.0, -90.0, -91.0], [-120.0, -121.0, -119.0, -300.0], [15.0, 14.0, 16.0, -16.0]])
    # with exponents of up to 400 a half step of the logit's product is 400 half steps of the result
    rel = 2 * (600 + 24) * ref.HALF
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.tensor([-5.0, 0.0, 0.0, 0.0])):
            want, w = ref.route(l, 2, score=score, bias=bias)
            ids, got = mxq.mxq_route_experts(l.to(DEV), 2, score=score, bias=None if bias is None else bias.to(DEV))
            assert torch.equal(ref.host(ids), want)
            ref.check_values(got, w, w.abs() * rel, "weights")
            assert torch.allclose(got.sum(1).cpu(), torch.ones(4), atol=1e-6)
            dw = torch.tensor([[1.0, -2.0]]).repeat(4, 1)
            grad, size = ref.route_backward(dw, l, want, score=score)
            d = mxq.mxq_route_experts_backward(dw.to(DEV), l.to(DEV), ids, score=score)
            ref.check_values(d, grad, size * rel, "dlogits")


def test_route_scores_next_to_each_other():
    """Biased scores that differ by less than fp32 resolves are told apart as 64 bits tell them."""
    g = gen(9)
    E = 64
    for score in ("sigmoid", "softmax"):
        l = (0.5 * torch.randn(200, E, generator=g)).float()
        p = torch.tensor(ref.scores(l[:1], score), dtype=torch.float64)
        bias = (1.0 - p[0]).float()          # the first token's keys all lie within a step of 1
        l[1:100] = l[0]
        l[1:100] += torch.randint(-1, 2, (99, E), generator=g) * 2.0 ** -22
        check(l, 6, score=score, bias=bias)
        check(l, 6, score=score, bias=bias, n_groups=8, top_groups=3, group_top=2)
    check(torch.linspace(30, 90, E)[None].repeat(3, 1), 6, score="sigmoid")                       # saturated: by the logits
    check(torch.linspace(30, 90, E)[None].repeat(3, 1), 6, score="sigmoid", bias=torch.zeros(E))  # by the scores: many are 1


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (256, 16), (96, 6), (32, 2), (512, 4), (80, 16)])
def test_route_few_next_to_each_other(E, groups, score):
    """Clusters of 2 to 20 keys, or of two groups, that fp32 does not tell apart, and nothing else near: at the last choice, before
    it and behind it.  The keys of a token differ from the first token's by a few steps of fp32."""
    g = gen(E + groups)
    l = (0.5 * torch.randn(1, E, generator=g)).repeat(40, 1)
    p = torch.tensor(ref.scores(l[:1], score), dtype=torch.float64)[0]
    l[1:] += torch.randint(-2, 3, (39, E), generator=g) * 2.0 ** -22
    mask = torch.arange(40) % 7 != 3
    for cluster in (2, 15, 16, 17, 20):
        place = torch.empty(E, dtype=torch.long)
        place[torch.randperm(E, generator=g)] = torch.arange(E) // cluster
        bias = (1 + 0.02 * place - p).float()
        for k in (1, 7, 15):
            check(l, k, score=score, bias=bias, mask=mask)
    size = E // groups
    for width in (2, groups):
        inside = torch.rand(E // groups, generator=g).repeat(groups)          # the groups of a cluster are alike
        bias = (1 + 0.02 * (torch.arange(E) // size // width) + 0.3 * inside - p).float()
        for top in (1, (groups + 1) // 2):
            for group_top in (1, 2):
                check(l, min(5, size), score=score, bias=bias, mask=mask, n_groups=groups, top_groups=top, group_top=group_top)
    if score == "sigmoid":   # groups of equal logits, which rank by their scores
        l = l.view(40, groups, size)[:, :1].repeat(1, groups, 1) + torch.randint(-2, 3, (40, groups, size), generator=g) * 2.0 ** -22
        check(l.reshape(40, E), min(5, size), score=score, n_groups=groups, top_groups=(groups + 1) // 2, group_top=2)


def test_route_biases_of_the_lowest_value():
    """Experts that a bias of about the lowest number puts last, also in groups whose two add up to less than that."""
    g = gen(21)
    E, low = 64, torch.finfo(FP32).min
    l = logits_of(30, E, 22)
    l[3:6, 5:20] = -INF
    for score in ("softmax", "sigmoid"):
        for part in (slice(8, 60), slice(0, 64), slice(17, 24)):
            bias = 0.1 * torch.randn(E, generator=g)
            bias[part] = low * (1 - 0.25 * torch.rand(E, generator=g)[part])
            bias[20:26] = low
            for k, how in ((8, {}), (20, {}), (8, {"n_groups": 8, "top_groups": 5, "group_top": 2}), (6, {"n_groups": 8, "top_groups": 2}),
                           (3, {"n_groups": 16, "top_groups": 9, "group_top": 2})):
                check(l, k, score=score, bias=bias, **how)


def test_route_values_that_are_not_finite():
    """A NaN is chosen last of those that are open; +Inf first; nothing else of the batch changes."""
    l = logits_of(20, 40, 11)
    plain, w = mxq.mxq_route_experts(l.to(DEV), 4)
    l[3, 7] = math.nan
    l[5, :] = math.nan
    l[9, 21] = INF
    l[11, :38] = -INF
    l[11, 38] = math.nan
    for score in ("softmax", "sigmoid"):
        ids, got = mxq.mxq_route_experts(l.to(DEV), 4, score=score)
        keep = [t for t in range(20) if t not in (3, 5, 9, 11)]
        assert torch.equal(ids[keep], plain[keep])
        assert 7 not in ids[3].tolist() and ids[5].tolist() == [0, 1, 2, 3] and ids[9, 0] == 21
        assert ids[11].tolist() == [39, 38, -1, -1] and bool(torch.isnan(got[5]).all())
        if score == "softmax":
            assert torch.equal(got[keep], w[keep])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_route_masks_of_the_lowest_value(dtype):
    """Logits of the type's lowest value are open and last; a token that has no others shares its weight out evenly."""
    l = logits_of(30, 96, 19, dtype)
    low = torch.finfo(dtype).min
    l[:, 10:80] = low
    l[4] = low
    l[5, 3:] = low
    for score in ("softmax", "sigmoid"):
        for how in ({}, {"n_groups": 8, "top_groups": 8}, {"n_groups": 8, "top_groups": 2}):
            want, _ = ref.route(l, 5, score=score, **how)
            ids, w = mxq.mxq_route_experts(l.to(DEV), 5, score=score, **how)
            assert torch.equal(ref.host(ids), want)
            assert bool(torch.isfinite(w).all()) and torch.allclose(w.sum(1).cpu(), torch.ones(30), atol=1e-6)
            assert torch.allclose(w[4].cpu(), torch.full((5,), 0.2))
            d = mxq.mxq_route_experts_backward(w, l.to(DEV), ids, score=score)
            assert bool(torch.isfinite(d).all())


def test_route_backward_of_ids_out_of_range_and_named_twice():
    """Ids that are no expert's count nothing; an expert named twice gets the sum."""
    l = logits_of(6, 20, 12)
    ids = torch.tensor([[3, 3], [-1, 5], [20, 4], [2 ** 31 - 1, -7], [0, 19], [-1, -1]], dtype=torch.int32)
    dw = torch.randn(6, 2, generator=gen(13))
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            got = mxq.mxq_route_experts_backward(dw.to(DEV), l.to(DEV), ids.to(DEV), score=score, renormalize=renormalize)
            want, size = ref.route_backward(dw, l, ids, score=score, renormalize=renormalize)
            ref.check_values(got, want, size * 2 * REL, "dlogits")


def test_route_backward_against_differences():
    """Along directions, against differences of the forward call with the choice held: fp32 weights of at most 2.5 are off
    by 2^-23 of 3 terms, divided by 2 h with h = 2^-8; the third derivative adds a few h^2."""
    l, v = logits_of(3, 12, 14), torch.randn(3, 12, generator=gen(15))
    dw = torch.randn(3, 3, generator=gen(16))
    h = 2.0 ** -8
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            how = dict(score=score, renormalize=renormalize, scale=2.5)
            ids, _ = mxq.mxq_route_experts(l.to(DEV), 3, **how)
            # a bias that settles the choice whatever the step does
            f = lambda x: sum(float((ref.f64(mxq.mxq_route_experts(x[t:t + 1].to(DEV), 3, bias=lift[t], **how)[1]) * order[t]).sum()) for t in range(3))
            lift, order = [], []
            for t in range(3):
                b = torch.zeros(12)
                for j, e in enumerate(ids[t].tolist()):
                    b[e] = 30.0 - 10 * j
                lift.append(b.to(DEV))
                order.append(dw[t].double())
            got = float((ref.f64(mxq.mxq_route_experts_backward(dw.to(DEV), l.to(DEV), ids, **how)) * v.double()).sum())
            assert abs((f(l + h * v) - f(l - h * v)) / (2 * h) - got) < 100 * h * h + 9 * 2.5 * 2.0 ** -23 * 3 / h


def test_route_of_nothing_and_its_own_buffers():
    ids, w = mxq.mxq_route_experts(torch.zeros(0, 8, device=DEV), 2)
    assert ids.shape == w.shape == (0, 2)
    assert mxq.mxq_route_experts_backward(w, torch.zeros(0, 8, device=DEV), ids).shape == (0, 8)
    with pytest.raises(mxq.MxqError):
        mxq.mxq_route_experts(torch.zeros(2, 8, device=DEV), 9)
    with pytest.raises(mxq.MxqError):
        mxq.mxq_route_experts(torch.zeros(2, 8, device=DEV), 3, n_groups=4, top_groups=1)
    l = logits_of(10, 24, 17).to(DEV)
    ids, w = torch.full((10, 3), 9, dtype=torch.int32, device=DEV), torch.zeros(10, 3, device=DEV)
    wide = torch.full((12, 30), 5.0, device=DEV)
    assert mxq.mxq_route_experts(l, 3, ids=ids, weights=w)[0] is ids
    mxq.mxq_route_experts_backward(w, l, ids, dlogits=wide[1:11, 2:26])
    inside = torch.zeros(12, 30, dtype=torch.bool)
    inside[1:11, 2:26] = True
    assert bool((wide.cpu()[~inside] == 5.0).all())


def test_route_feeds_the_sort_in_a_captured_graph():
    """Routed, sorted, and the gradient back, replayed with other logits and masks."""
    bias = 0.1 * torch.randn(48, generator=gen(1)).to(DEV)
    l, mask = logits_of(70, 48, 2).to(DEV), torch.ones(70, dtype=torch.bool, device=DEV)

    def step(l, mask):
        ids, w = mxq.mxq_route_experts(l, 6, bias=bias, score="sigmoid", n_groups=8, top_groups=4, group_top=2, mask=mask)
        return (ids, w, *mxq.mxq_sort_experts(ids, 48), mxq.mxq_route_experts_backward(w, l, ids, score="sigmoid"))

    step(l, mask)
    sl, sm = l.clone(), mask.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(sl, sm)
    for k in range(4):
        sl.copy_(l.roll(k, 1) + k)
        sm.copy_(torch.arange(70, device=DEV) % (k + 2) != 0)
        want = step(sl, sm)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
        assert int(out[2][-1]) == int(sm.sum()) * 6
