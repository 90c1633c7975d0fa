"""Which kernel a product of FP8 operands takes (csrc/product_choice.h), on the host."""
import os
import shutil
import subprocess

import pytest

from tests.product_sizes import CASES, KERNELS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "microscaling_weight_quantization_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "product_choice.h"
int main() {
  long mode, fast, fed, I, J, experts;
  while (scanf("%ld %ld %ld %ld %ld %ld", &mode, &fast, &fed, &I, &J, &experts) == 6)
    printf("%d\n", (int)mxq_host::choose_kernel((mxq_host::Mode)mode, fast, fed, I, J, experts));
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cpp").write_text(PROGRAM)
    subprocess.check_call([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "choice.cpp"), "-o", str(d / "choice")])

    def many(cases):
        """[(mode, fast, fed, I, J, experts)] -> [kernel name]"""
        text = "\n".join(" ".join(str(int(v)) for v in (("y", "dx", "dw").index(c[0]), *c[1:])) for c in cases)
        out = subprocess.run([str(d / "choice")], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [KERNELS[int(k)] for k in out]

    return many


def test_sizes_reach_the_kernels_they_are_meant_for(choose):
    got = choose([(c.mode, c.fast, c.fed, c.I, c.J, c.experts) for c in CASES])
    assert [f"{c} took {k}" for c, k in zip(CASES, got) if k != c.kernel] == []


def test_every_kernel_is_reached_in_every_mode():
    for mode, kernels in (("y", KERNELS), ("dx", KERNELS), ("dw", ("kExact", "kExactCarried"))):
        for k in kernels:
            cases = [c for c in CASES if c.mode == mode and c.kernel == k]
            assert cases, (mode, k)
            if k.startswith(("kTiles", "kCarried", "kExact", "kFewRows64")):
                assert any(not c.experts for c in cases), (mode, k)
            if k.startswith(("kTiles", "kCarried", "kExact")):
                assert any(c.experts for c in cases), (mode, k)


def test_alignment_of_the_sizes():
    """A fed case's contiguous axes end on whole 16 bytes."""
    for c in CASES:
        axes = {"y": (c.R,), "dx": (c.R, c.J), "dw": (c.I, c.J)}[c.mode]
        assert not c.fed or all(a % 16 == 0 for a in axes), c


def test_the_smallest_batches_take_the_few_rows_kernels(choose):
    """One token by expert is fewer rows than experts: as many more tokens are, it is few rows."""
    for experts, top_k, J in ((48, 6, 1024), (48, 6, 2048), (128, 8, 768), (8, 2, 14336)):
        for mode, fast in (("y", True), ("y", False), ("dx", False)):
            cases = [(mode, fast, True, t * top_k, J, experts) for t in (1, 2, 3, 4, 6, 9)]
            assert set(choose(cases)) == {"kFewRows16"}, (experts, J, mode, fast)
    # one weight: between the sizes whose few-rows workgroups fit the card and those whose tiles fill it
    for J in (8192, 16384, 20480, 24576, 28672):
        assert set(choose([("y", True, True, rows, J, 0) for rows in (1, 4, 8)])) == {"kFewRows16"}, J
        assert set(choose([("y", False, True, rows, J, 0) for rows in (1, 4, 16)])) == {"kFewRows16"}, J
