"""The attention kernels' bounded waits leave no warp behind.  Where warps meet at a named barrier
while each of them has waits of its own, one whose wait ran out still comes to the barriers at which
the others, whose waits ended in time, would wait for it: the sources, on the CPU, and the two forms
that they have, on the GPU."""
import ctypes
import os
import re

import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn
from test_abi import fake_addresses, lib  # noqa: F401  (fixture)
from test_layer_dependents import CSRC, kernels

KERNELS = {name: code for f in ("attention_prefill.cu", "attention_backward.cu", "attention_decode.cu")
           for name, code in kernels(open(os.path.join(CSRC, f)).read())}
BARRIER = re.compile(r"bar\.sync|bar_sync\(|bar_agree\(")


def loops(code):
    """(body, what follows) of a function's loops, outer ones too."""
    for m in re.finditer(r"\bfor \([^{;]*;[^{;]*;[^{;]*\{", code):
        depth, end = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[end], 0)
            end += 1
        yield code[m.end():end - 1], code[end:]


MEETING = [(name, *loop) for name, code in KERNELS.items() for loop in loops(code)
           if BARRIER.search(loop[0]) and "mbar_wait" in loop[0]]


def test_the_loops_are_found():
    assert {m[0] for m in MEETING} == {"keys_kernel", "decode_kernel"}


@pytest.mark.parametrize("name,body,behind", MEETING, ids=[m[0] for m in MEETING])
def test_a_warp_whose_wait_ran_out_meets_the_others(name, body, behind):
    """It says so at a barrier that asks all and is the next one behind every wait; or it goes on to
    the barriers of all steps that are left, where every step has one, its first thing."""
    strip = lambda t: re.sub(r"//[^\n]*", "", t).lstrip()  # noqa: E731
    waits = [m.end() for m in re.finditer(r"ok = mbar_wait_warp_cycles\([^;]*;", body)]
    assert waits
    drains = re.match(r"if \(!ok\)\s*while \(\+\+i < n\) bar_sync\(", strip(behind))
    for at in waits:
        told = re.match(r"if \(!ok\) \{\s*(attn::)?bar_agree\([^;]*false\);\s*break;\s*\}",
                        strip(body[at:]))
        if told:
            rest = strip(body[at:])[told.end():]
            assert BARRIER.search(rest).group() == "bar_agree(", name
        else:
            assert drains and len(BARRIER.findall(body)) == 1, name
            assert BARRIER.search(body).start() < min(waits) and "continue" not in body


def test_every_way_out_waits_for_the_kernel_beside():
    """The queries' kernel of the gradients starts beside the keys' one, and its end stands for the
    end of both: whichever way a CTA leaves, it has waited for the grid before."""
    code = re.sub(r"//[^\n]*", "", KERNELS["queries_kernel"])
    assert "return;" in code
    ways = [code[:m.start()] for m in re.finditer(r"\breturn;", code)] + [code.rstrip()[:-1]]
    for way in ways:
        last = [x.strip() for x in way.rstrip().rstrip(";").split(";")][-1]
        assert last.split("{")[-1].strip() == "grid_wait()", way[-120:]


def test_the_join_knows_its_rows_before_any_wait():
    """The kernel that joins a prompt's parts writes to the rows that the first part names.  They are
    named before the first wait that could run out, or the join would go by unset memory."""
    code = re.sub(r"//[^\n]*", "", KERNELS["prefill_kernel"])
    softmax = code[code.index("setmaxnreg.inc"):]
    assert len(re.findall(r"a\.dest\[", softmax)) == 1
    assert softmax.index("a.dest[") < softmax.index("mbar_wait") and softmax.index("a.dest[") < \
        softmax.index("take(")


ALLOCATING = [(name, code) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh"))
              for name, code in kernels(open(os.path.join(CSRC, f)).read())
              if "tmem_alloc" in code and "grid_release_next()" in code]


def test_dependents_start_behind_the_allocation_of_tensor_memory():
    """A dependent may take an SM's tensor memory and then wait for this grid's end, so no kernel lets
    it start before all of its own CTA's columns are there."""
    assert {n for n, _ in ALLOCATING} >= {"prefill_kernel", "pair_gemm_kernel", "split_gemm_kernel"}
    for name, code in ALLOCATING:
        code = re.sub(r"//[^\n]*", "", code)
        at, release = code.index("tmem_alloc"), code.index("grid_release_next()")
        assert "__syncthreads();" in code[at:release], name


@fake_addresses
def test_the_hook_refuses(lib):  # noqa: F811
    f = hook(lib)
    at = ctypes.c_void_p(0x100000000)
    for bad in ((2, 1, 0, 4, 1, 100, at), (0, 16, 0, 4, 1, 100, at), (0, 1, -1, 4, 1, 100, at),
                (0, 1, 0, 0, 1, 100, at), (0, 1, 0, 1001, 1, 100, at), (1, 1, 0, 4, 0, 100, at),
                (0, 1, 0, 4, 1, -1, at), (0, 1, 0, 4, 1, 2 * 10 ** 9 + 1, at), (0, 1, 0, 4, 1, 100, None)):
        assert f(*bad, None) == 1, bad


def hook(library):
    f = library.gdn_testing_group_wait
    f.argtypes = [ctypes.c_int32, ctypes.c_uint32] + [ctypes.c_int32] * 3 + [ctypes.c_int64] + \
        [ctypes.c_void_p] * 2
    f.restype = ctypes.c_int
    return f


@pytest.mark.gpu
@pytest.mark.parametrize("late", [0, 1, 4, 5, 15])
@pytest.mark.parametrize("asks,steps,part", [(0, 1, 1), (0, 7, 1), (1, 1, 1), (1, 9, 4), (1, 8, 4)])
def test_no_warp_waits_for_one_that_left(gdn_lib, asks, steps, part, late):
    f = hook(gdn_lib.load())
    for step in range(steps):
        left = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        assert f(asks, late, step, steps, part, 2_000_000, left.data_ptr(),
                 torch.cuda.current_stream().cuda_stream) == 0
        # the others: at the barrier of the part's last step, or not at all
        end = min(step - step % part + part, steps) - 1 if asks and late else steps
        assert left.tolist() == [step if late >> w & 1 else end for w in range(4)], step
        assert gdn.device_status() == (5 if late else 0)
