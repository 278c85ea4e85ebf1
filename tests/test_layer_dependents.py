"""Kernels that wait for the grid before them (grid_wait) are resident while
that grid still writes: what they read of global memory is not read-only for
their lifetime.  Their sources therefore use no non-coherent load and promise
the compiler no read-only pointer."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "hybrid_linear_attention_deltanet_gb300", "csrc")


def kernels(text):
    """(name, signature and body) of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        body = text.index("{", text.index(")", re.compile(r"\w+_kernel\s*\(").search(
            text, m.end()).end()))
        depth, end = 0, body
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        name = re.search(r"(\w+_kernel)\s*\(", text[m.start():body]).group(1)
        yield name, text[m.start():end]


DEPENDENT = [(os.path.basename(p), name, code)
             for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
             for name, code in kernels(open(p).read()) if "grid_wait()" in code]


def test_the_dependents_are_found():
    assert {n for _, n, _ in DEPENDENT} >= {"pair_gemm_kernel", "split_gemm_kernel",
                                            "sum_parts_kernel", "norm_dw_kernel"}


@pytest.mark.parametrize("file,name,code", DEPENDENT, ids=[d[1] for d in DEPENDENT])
def test_dependents_load_coherently(file, name, code):
    assert "__ldg" not in code and "global.nc" not in code, file
    assert "__restrict__" not in code, file
