"""The layer of examples/expert_layer.py, forward, backward and for one token, against fp32.

E4M3 rounds by at most 2^-4 of a value, evenly spread about a third of that on
average in the root mean square of a dot product's independent roundings: an operand
quantized once is off by about 2^-4 / sqrt(3) = 0.036 of its norm and so is a product
with one such operand.  y passes two quantized operands, doubled by the square of the
activation between them, and the gradients up to four: 0.2 bounds them all.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [(96, 8, 2, 256, 384), (37, 5, 3, 200, 136)])
def test_expert_layer(sizes):
    from examples import expert_layer
    args = [v for n, s in zip(("tokens", "experts", "top-k", "hidden", "inner"), sizes) for v in ("--" + n, str(s))]
    off = expert_layer.main(args)
    assert set(off) == {"y", "dx", "dweights", "dup", "ddown", "token"}
    assert all(v < 0.2 for v in off.values()), off
