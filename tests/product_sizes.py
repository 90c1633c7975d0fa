"""Sizes that reach each kernel of the FP8 products, and the kernel that each is meant
to reach.  A host test evaluates the library's own rule on them, so that a change
of the rule cannot leave a kernel untested; the GPU tests run them.

out[I, J] = sum over R; y is [tokens, N] over K, dx [tokens, K] over N, dw [N, K] over
tokens.  `fed`: rows begin at multiples of 16 bytes and end on them.  With experts the
rows I (R for dw) are sorted by expert.
"""
from typing import NamedTuple


class Case(NamedTuple):
    mode: str
    fast: bool
    fed: bool
    I: int
    R: int
    J: int
    experts: int
    kernel: str

    def __str__(self):
        return "-".join((self.mode, "fast" if self.fast else "fp32", "fed" if self.fed else "odd", f"{self.I}x{self.R}x{self.J}",
                         f"{self.experts}e" if self.experts else "one", self.kernel))


def _both(*a):
    return [Case("y", *a), Case("dx", *a)]


CASES = (
    # few rows: 16, 32 or 64 a workgroup, of eight waves or, where they fill the card, of four
    _both(False, True, 9, 400, 2000, 0, "kFewRows16") + _both(False, True, 7, 272, 24592, 0, "kFewRows16")
    + _both(True, True, 9, 400, 2000, 0, "kFewRows16") + [Case("y", True, True, 7, 272, 24592, 0, "kFewRows16")]
    + _both(False, True, 30, 400, 2000, 0, "kFewRows32") + _both(False, True, 30, 272, 24592, 0, "kFewRows32")
    + _both(True, True, 30, 400, 2000, 0, "kFewRows32")
    + _both(False, True, 150, 400, 2000, 0, "kFewRows64") + _both(False, True, 120, 272, 4096, 3, "kFewRows64")
    + _both(True, True, 150, 400, 2000, 0, "kFewRows64") + _both(True, True, 120, 272, 4096, 3, "kFewRows64")
    + _both(False, False, 9, 401, 2001, 0, "kFewRows16") + _both(True, False, 9, 401, 2001, 0, "kFewRows16")
    + _both(False, False, 30, 401, 2001, 0, "kFewRows32") + _both(True, False, 30, 401, 2001, 0, "kFewRows32")
    + _both(False, False, 150, 401, 2001, 0, "kFewRows64") + _both(True, False, 150, 401, 2001, 0, "kFewRows64")
    # tiles of FP8 sums: three blocks of codes byte by byte, four and eight of them in words
    + _both(True, True, 300, 272, 4304, 0, "kTiles128") + _both(True, True, 300, 512, 4304, 0, "kTiles128")
    + _both(True, True, 300, 1000 // 16 * 16, 4304, 0, "kTiles128") + _both(True, True, 700, 400, 2064, 4, "kTiles128")
    + _both(True, True, 520, 272, 13200, 0, "kTiles256") + _both(True, True, 520, 512, 13200, 0, "kTiles256")
    + _both(True, True, 1500, 400, 5136, 3, "kTiles256")
    # rows of any alignment through registers
    + _both(True, False, 300, 275, 7001, 0, "kCarried") + _both(True, False, 700, 400, 3001, 4, "kCarried")
    # sums in fp32
    + _both(False, True, 300, 272, 4304, 0, "kExact") + _both(False, True, 700, 400, 2064, 4, "kExact")
    + _both(False, False, 300, 275, 7001, 0, "kExactCarried") + _both(False, False, 700, 400, 3001, 4, "kExactCarried")
    + [Case("dw", False, True, 272, 600, 400, 0, "kExact"), Case("dw", False, True, 272, 600, 400, 4, "kExact"),
       Case("dw", False, False, 273, 600, 401, 0, "kExactCarried"), Case("dw", False, False, 273, 600, 401, 4, "kExactCarried")]
)

KERNELS = ("kFewRows16", "kFewRows32", "kFewRows64", "kTiles128", "kTiles256", "kCarried", "kExact", "kExactCarried")


def offsets_of(rows: int, experts: int):
    """Ragged shares: the second expert has none, and the last rows belong to nobody."""
    if not experts:
        return None
    weights = [0 if e == 1 else 2 * e + 3 for e in range(experts)]
    out = [0]
    for w in weights:
        out.append(out[-1] + w * (rows - rows // 20) // sum(weights))
    return out
