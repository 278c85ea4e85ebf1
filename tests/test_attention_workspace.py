"""The gradients' workspace: one that is sized for the largest problem serves all smaller ones (the
sizes, on the CPU; the calls, on the GPU, with the bits of the library's own scratch)."""
import random

import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn
from test_abi import lib  # noqa: F401  (fixture)


def size(*args):
    return gdn.load().gdn_attention_prefill_backward_workspace_size(*args)


@pytest.mark.parametrize("varlen", [0, 1])
@pytest.mark.parametrize("H,kv,d", [(16, 4, 128), (6, 2, 64), (1, 1, 128), (128, 1, 64), (64, 64, 128)])
def test_sizes_grow_with_the_problem(lib, varlen, H, kv, d):  # noqa: F811
    last = 0
    for T in (1, 17, 128, 300, 700, 1024, 1500, 2048, 4096, 6000, 8192, 16384, 65536):
        now = size(1, T, T, varlen, H, kv, d)
        assert now >= last, T
        last = now
    rng = random.Random(H)
    for _ in range(3000):
        small = [int(2 ** rng.uniform(0, top)) for top in (8, 15, 15)]
        large = [n + rng.choice([0, 0, 1, n, 10 * n]) for n in small]
        assert size(*small, varlen, H, kv, d) <= size(*large, varlen, H, kv, d), (small, large)


@pytest.mark.gpu
@pytest.mark.parametrize("H,kv,d", [(16, 4, 128), (3, 1, 64)])
def test_one_workspace_for_the_longest(gdn_lib, H, kv, d):
    rng, most = random.Random(d), 8192
    nbytes = gdn.attention_prefill_backward_workspace_size(4, most, H, kv, d, varlen=True)
    ws = torch.full((nbytes + 256,), 255, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0
    for T in (8192, 4096, 1024, 2048, 300, 17, 1, rng.randint(1, most), rng.randint(1, most)):
        g = torch.Generator(device="cuda").manual_seed(T)
        q, dout, k, v = (torch.randn(T, h, d, generator=g, device="cuda").to(torch.bfloat16)
                         for h in (H, H, kv, kv))
        cuts = sorted(rng.randint(0, T) for _ in range(rng.randint(0, 3)))
        c = torch.tensor([0, *cuts, T], dtype=torch.int32, device="cuda")
        out, lse = gdn.attention_prefill(q, k, v, c)
        want = gdn.attention_prefill_backward(q, k, v, out, lse, dout, c)
        got = gdn.attention_prefill_backward(q, k, v, out, lse, dout, c, workspace=ws[:nbytes])
        assert all(torch.equal(want[n], got[n]) for n in want), T
        # and one of its own size
        own = gdn.attention_prefill_backward_workspace_size(len(c) - 1, T, H, kv, d, varlen=True)
        got = gdn.attention_prefill_backward(q, k, v, out, lse, dout, c, workspace=ws[:own])
        assert all(torch.equal(want[n], got[n]) for n in want), T
    assert (ws[nbytes:] == 255).all() and gdn.device_status() == 0
