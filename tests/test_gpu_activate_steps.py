"""How many roundings the activation and its gradients take before the one to E4M3.  A group of one element has the
smallest code S whose 448 2^S holds it, so the code of a value next to such a border tells on which side of it the kernel
took it: values within 40 half steps of a border, and codes that may differ only where a derived number of half steps allows it.

Half steps (2^-24 of the value) that the kernel takes, with z the logistic function's argument:
  t = exp(-z): the exponential 2, what is left of its argument (at most 1/2, rounded twice) 0.35; 1 + t: 1; its reciprocal 2.
  p is 1 / (1 + t), q = 1 - p is t / (1 + t), one product more; t weighs at most 1 in either: 2.35 + 1 + 2 + 1 = 6.35.
  silu: g p 1, times up or da 1: 8.35.  Its slope p + g p q: (6.35 + 1) + 6.35 + 1 = 14.7 for the second term, the sum 1,
  da up and its product with the slope 2: 17.7 of the sum of magnitudes.
  gelu: z = c (g + k g^3) with both constants rounded is off by 7 of itself, which p takes over times |z| q: 7 |z| more.
  The slope p + g p q c (1 + 3 k g^2): p q has z's error once, (p + q = 1); c, its product, 3 k, g^2, their product, the sum and
  the last product 7: 17.7 + 7 + 7 |z|.
"""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from tests import between_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
N = 30000


def steps(act, g):
    """(forward, slope) half steps for gates g."""
    z = g.abs() if act == "silu" else (ref.KGELU * (g + 0.044715 * g ** 3)).abs()
    more = 0.0 if act == "silu" else 7.0
    return 8.35 + more * z + 1e-3, 17.7 + more * (1 + z) + 1e-3


def next_to_a_border(size, g):
    """fp32 factors that bring `size` (64 bits, not 0) within 40 half steps of 448 2^S."""
    want = 448 * 2.0 ** torch.randint(-3, 4, size.shape, generator=g).double()
    want *= 1 + 40 * ref.HALF * (2 * torch.rand(size.shape, generator=g).double() - 1)
    return (want / size).float()


def gates(act, seed):
    g = torch.Generator().manual_seed(seed)
    far = 20.0 if act == "silu" else 4.0
    x = (2 * torch.rand(N, generator=g) - 1) * far * torch.rand(N, generator=g) ** 2
    return torch.where(x.abs() < 1e-3, torch.tensor(0.5), x), g


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("by_rows", [True, False])
def test_activation_half_steps(act, by_rows):
    x, g = gates(act, 1)
    a = ref.act(act, x.double())[0]
    up = next_to_a_border(a.abs(), g)
    want = a * up.double()
    off = want.abs() * steps(act, x.double())[0] * ref.HALF
    if by_rows:
        q, c = mxq.mxq_activate_fp8_group128(x[:, None].to(DEV), up[:, None].to(DEV), act)
        ref.check_rows(q, c, want[:, None], off[:, None])
    else:
        _, _, q, c = mxq.mxq_activate_fp8_group128_row_col(x[None].to(DEV), up[None].to(DEV), act)
        ref.check_cols(q, c, want[None], off[None])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("half", ["gate", "up"])
def test_activation_gradient_half_steps(act, half):
    x, g = gates(act, 2)
    a, d, size, _ = ref.act(act, x.double())
    up = torch.exp2(torch.randint(-2, 3, (N,), generator=g).float())     # its product with da is exact
    da = next_to_a_border((d * up if half == "gate" else a).abs().clamp(min=1e-6), g)
    want = torch.cat((da.double() * up.double() * d, da.double() * a))
    forward, slope = steps(act, x.double())
    off = torch.cat(((da.double() * up.double()).abs() * size * slope, (da.double() * a).abs() * forward)) * ref.HALF
    _, _, q, c = mxq.mxq_activate_fp8_group128_backward(da[None].to(DEV), x[None].to(DEV), up[None].to(DEV), act)
    ref.check_cols(q, c, want[None], off[None])
