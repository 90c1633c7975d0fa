"""The gradient of the router's logits where a token has no expert at all: zeros, whatever its logits hold."""
import math

import pytest
import torch

import microscaling_weight_quantization_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("E,k", [(48, 6), (50, 6), (300, 16), (64, 20), (512, 100)])
def test_route_gradient_of_masked_tokens(E, k, renormalize, score, dtype):
    """Padded places that hold NaN or infinities; the other tokens' gradients are those of a batch without them."""
    g = torch.Generator().manual_seed(E + k)
    clean = torch.randn(37, E, generator=g).to(dtype)
    l, mask = clean.clone(), torch.ones(37, dtype=torch.bool)
    for t, v in ((1, math.nan), (4, math.inf), (17, -math.inf), (36, math.nan)):
        l[t] = v
        mask[t] = False
    l[20, 3], l[21, E - 1], l[22, 5] = math.nan, math.inf, -math.inf
    mask[20:23] = False
    how = dict(score=score, renormalize=renormalize, scale=2.5)
    ids, w = mxq.mxq_route_experts(l.to(DEV), k, mask=mask.to(DEV), **how)
    assert bool((ids[~mask] == -1).all()) and bool((w[~mask] == 0).all())
    dw = torch.randn(37, k, generator=g)
    dw[4, 0] = math.nan                     # a gradient of a weight that is not there
    got = mxq.mxq_route_experts_backward(dw.to(DEV), l.to(DEV), ids, **how).cpu()
    assert bool((got[~mask] == 0).all())
    want = mxq.mxq_route_experts_backward(dw.to(DEV), clean.to(DEV), ids, **how).cpu()
    assert torch.equal(got[mask], want[mask]) and bool(torch.isfinite(got).all()) and bool((got[mask] != 0).any())
    # ids that are no expert's are no choice either
    other = torch.where(mask[:, None], ids.cpu(), torch.randint(E, 2 ** 31 - 1, (37, k), generator=g).int())
    assert torch.equal(mxq.mxq_route_experts_backward(dw.to(DEV), l.to(DEV), other.to(DEV), **how).cpu(), got)
