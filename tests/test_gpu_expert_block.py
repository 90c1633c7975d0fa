"""The norm, the routing, the activation and the products together, as examples/expert_block.py uses them, forward, backward
and for a few tokens, against fp32; and the same step captured into a graph.

E4M3 rounds by at most 2^-4 of a value, evenly spread about a third of that in the root mean square of a dot
product's independent roundings: an operand quantized once is off by about 2^-4 / sqrt(3) = 0.036 of its norm and
so is a product with one such operand.  y passes two quantized operands, the first of them in two factors of a
product; the gradients pass up to four: 0.2 bounds them all.  The router's gradient passes the products' error in
differences p_j - sum p p / sum, which are of the size of what is taken apart: 0.2 as well.  The residual is a sum
in fp32; a few tokens alone take other kernels for the products, whose sums in the matrix cores' own FP8 may be off by 2^-10
of the sum of magnitudes -- up to 2^-10 sqrt(K) of a result's norm, 0.02 at K = 400 -- twice.
"""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [(96, 8, 2, 1, 256, 384), (150, 16, 3, 4, 256, 128), (37, 6, 3, 2, 200, 136)])
def test_expert_block(sizes):
    from examples import expert_block
    names = ("tokens", "experts", "top-k", "groups", "hidden", "inner")
    off = expert_block.main([v for n, s in zip(names, sizes) for v in ("--" + n, str(s))])
    assert set(off) == {"y", "residual", "dx", "dnorm", "drouter", "dup", "ddown", "tokens"}
    assert off.pop("residual") < 1e-6
    assert off.pop("tokens") < 0.05, off
    assert all(v < 0.2 for v in off.values()), off


def test_expert_block_captured():
    """A whole step in a graph, replayed with other inputs and masks: the bits of the eager step."""
    from examples import expert_block
    block = expert_block.ExpertBlock(8, 256, 128, 3, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    draw = lambda dtype: torch.randn(70, 256, generator=g, device="cuda").to(dtype)

    def step(x, residual, dy, ds, mask):
        y, s, kept = block.forward(x, residual, mask, keep=True)
        return (y, s, kept[3], kept[4], *block.backward(dy, ds, kept)[:2])

    ins = [draw(torch.bfloat16), draw(torch.float32), draw(torch.bfloat16), draw(torch.float32),
           torch.ones(70, dtype=torch.bool, device="cuda")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*ins)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*ins)
    for k in range(4):
        for t in ins[:4]:
            t.copy_(draw(t.dtype) * (k + 1))
        ins[4].copy_(torch.arange(70, device="cuda") % (k + 2) != 0)
        want = step(*[t.clone() for t in ins])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
        assert bool((out[2][~ins[4]] == -1).all()) and bool((out[0][~ins[4]] == 0).all())


def test_two_streams_at_once():
    """Two blocks' steps on two streams of their own give what each gives alone."""
    from examples import expert_block
    block = expert_block.ExpertBlock(8, 256, 128, 3, 4)
    g = torch.Generator(device="cuda").manual_seed(6)
    ins = [[torch.randn(90, 256, generator=g, device="cuda").to(d) for d in (torch.bfloat16, torch.float32)] for _ in range(2)]
    alone = [block.forward(*i, keep=True)[:2] for i in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, (st, i) in enumerate(zip(streams, ins)):
            with torch.cuda.stream(st):
                got[k].append(block.forward(*i, keep=True)[:2])
    torch.cuda.synchronize()
    for k in range(2):
        for y, s in got[k]:
            assert torch.equal(y, alone[k][0]) and torch.equal(s, alone[k][1])
