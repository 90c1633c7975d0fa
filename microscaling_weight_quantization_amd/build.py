"""Build the gfx950 library (hipcc, in-tree).

``python -m microscaling_weight_quantization_amd.build`` writes
``libmxq.so`` next to this file, plus three variants of the same source used by
the build-variant tests: ``libmxq_fastmath.so`` (fast-math, denormals flushed),
``libmxq_o1.so`` (-O1) and ``libmxq_o0.so`` (-O0, no optimisation).  Every
step of the path is integer arithmetic, so all four builds must produce
identical bits.  The FP8 products, their quantizer and the expert routing
(``OBJECTS``) are compiled once, with -O3, and linked into all four.
``libmxq_shapes.so`` holds the access-shape reference kernels
(``csrc/shapes.hip``) that bench.py times beside the library's kernels.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "mxq.hip")
INCLUDE = os.path.join(ROOT, "include")
ARCH = "gfx950"

# Packed fp32 instructions are kept out of every build.
COMMON = ["--offload-arch=" + ARCH, "-std=c++17", "-fPIC", "-Wall",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + INCLUDE]

VARIANTS = {
    "libmxq.so": ["-O3"],
    "libmxq_fastmath.so": ["-O3", "-ffast-math", "-fgpu-flush-denormals-to-zero"],
    "libmxq_o1.so": ["-O1"],
    "libmxq_o0.so": ["-O0"],
    "libmxq_shapes.so": ["-O3"],
}
OBJECTS = ("group_quant", "product", "experts")
OBJECT_HEADERS = ("checks.h", "segments.h", "fastdiv.h", "product_choice.h")
SOURCES = {"libmxq_shapes.so": os.path.join(HERE, "csrc", "shapes.hip")}   # the others: SRC


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


def _compile(out: str, args, verbose: bool) -> str:
    tmp = out + f".tmp{os.getpid()}"
    cmd = [hipcc()] + COMMON + args + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, out)
    return out


def object_source(name: str) -> str:
    return os.path.join(HERE, "csrc", name + ".hip")


def build_object(name: str, verbose: bool = False) -> str:
    return _compile(os.path.join(HERE, name + ".o"), ["-O3", "-c", object_source(name)], verbose)


def build_one(name: str, flags, verbose: bool = False, objects=()) -> str:
    if name in SOURCES:
        return _compile(os.path.join(HERE, name), ["-shared"] + flags + [SOURCES[name]], verbose)
    return _compile(os.path.join(HERE, name), ["-shared"] + flags + list(objects) + [SRC], verbose)   # objects first: hipcc takes what follows a source for one


def build(variants=None, verbose: bool = False):
    names = list(VARIANTS) if variants is None else list(variants)
    with ThreadPoolExecutor(max(len(names), len(OBJECTS))) as ex:
        objects = list(ex.map(lambda n: build_object(n, verbose), OBJECTS)) if any(n not in SOURCES for n in names) else []
        return list(ex.map(lambda n: build_one(n, VARIANTS[n], verbose, objects), names))


def library_path(name: str = "libmxq.so") -> str:
    return os.path.join(HERE, name)


def stale(name: str = "libmxq.so") -> bool:
    lib = library_path(name)
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    if name in SOURCES:
        srcs = (SOURCES[name], os.path.join(INCLUDE, "mxq_shapes.h"))
    else:
        srcs = (SRC, os.path.join(INCLUDE, "mxq.h"), *(object_source(n) for n in OBJECTS),
                *(os.path.join(HERE, "csrc", h) for h in OBJECT_HEADERS))
    return any(os.path.getmtime(p) > t for p in srcs)


if __name__ == "__main__":
    for p in build(sys.argv[1:] or None, verbose=True):
        print(p)
