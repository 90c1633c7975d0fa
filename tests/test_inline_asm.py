"""Inline assembly of the kernels names the special registers that it writes."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "microscaling_weight_quantization_amd", "csrc")
SPECIAL = ("m0", "vcc", "exec")


def statements(text):
    """The text of each asm statement, parentheses balanced."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1]


def unnamed(text):
    """(statement, register) of each special register that an instruction writes and no clobber names."""
    out = []
    for s in statements(text):
        code, _, lists = s.partition(":")
        clobbers = lists.rsplit(":", 1)[-1]
        out += [(s, r) for r in SPECIAL if re.search(rf"[vs]_\w+\s+{r}\b", code) and f'"{r}"' not in clobbers]
    return out


def test_special_registers_are_named():
    files = glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h"))
    assert files and any(list(statements(open(f).read())) for f in files)
    for f in files:
        assert not unnamed(open(f).read()), f


def test_the_check_itself():
    assert unnamed('asm volatile("s_mov_b32 m0, %0" :: "s"(a) : "memory")')
    assert not unnamed('asm volatile("s_mov_b32 m0, %0" :: "s"(a) : "m0", "memory")')
