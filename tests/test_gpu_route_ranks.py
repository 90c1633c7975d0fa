"""Groups of experts that rank by the sum of two biased scores of opposite signs: the sum is as large as the scores, its
parts, each rounded once, are as large as the biases.  Choices are those of the definition in 64 bits all the same."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import between_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(logits, k, bias, score, groups, top):
    how = dict(score=score, n_groups=groups, top_groups=top, group_top=2)
    ids, _ = mxq.mxq_route_experts(logits.to(DEV), k, bias=bias.to(DEV), **how)
    want, _ = ref.route(logits, k, bias=bias, **how)
    wrong = (ref.host(ids) != want).any(1)
    assert not bool(wrong.any()), f"{int(wrong.sum())} of {len(wrong)} tokens, the first {int(torch.nonzero(wrong)[0])}"


def test_route_two_groups_by_hand():
    """Ranks 0.79919686 and 0.79919722; rounded keys put the first group first."""
    l = torch.tensor([[-0.45636314, -0.35839593, -0.45636368, -0.35839394]])
    bias = torch.tensor([16.0, -16.0, 16.0, -16.0])
    check(l, 2, bias, "sigmoid", 2, 1)
    assert mxq.mxq_route_experts(l.to(DEV), 2, bias=bias.to(DEV), score="sigmoid", n_groups=2, top_groups=1, group_top=2)[0].tolist() == [[2, 3]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("height", [16.0, 256.0, 1e4])
@pytest.mark.parametrize("E,groups,top,k", [(4, 2, 1, 2), (32, 16, 5, 6), (64, 8, 3, 8), (256, 8, 4, 8), (256, 16, 7, 5), (96, 6, 2, 4), (512, 2, 1, 12),
                                            (12, 4, 2, 3)])
def test_route_ranks_of_opposite_biases(E, groups, top, k, height, score):
    """In each group one expert far up and one far down, the rest further down still.  The two share a sum in other parts in every
    group; the sums lie apart by up to what a key of the bias's size is rounded by."""
    g = torch.Generator().manual_seed(E + groups + int(height))
    T, size = 150, E // groups
    first = torch.arange(groups) * size
    up = torch.randint(0, size, (groups,), generator=g)
    down = (up + torch.randint(1, size, (groups,), generator=g)) % size
    bias = torch.full((E,), -2 * height)
    bias[first + up], bias[first + down] = height, -height
    part = 0.3 + 0.4 * torch.rand(T, groups, generator=g).double()
    total = 0.8 * (1 + 4 * height * 2.0 ** -24 * torch.rand(T, groups, generator=g).double())
    a, b = part * total, (1 - part) * total
    to_logit = (lambda s: torch.log(s / (1 - s))) if score == "sigmoid" else torch.log
    l = torch.randn(T, E, generator=g) - 6
    l[:, first + up], l[:, first + down] = to_logit(a).float(), to_logit(b).float()
    check(l, k, bias, score, groups, top)
