"""What the attention layer's example prints is held to bounds, and the cache's 8-bit codes to the
rule's definition in 64 bits."""
import os
import re
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


def test_the_examples_errors(gdn_lib, capsys):
    """Both paths' outputs are rounded to e4m3 before the output projection, 2^-4 of each number at
    most, so two paths differ by 2^-3 at most where the attention agrees (bf16: within 2^-7, which
    moves few codes); keys and values in 8 bits are off by 2^-4 of themselves each, another 2^-3."""
    import attention_layer
    attention_layer.main()
    text = capsys.readouterr().out
    found = re.findall(r"^(\w+) cache: .* relative ([\d.e+-]+)", text, re.M)
    assert [t for t, _ in found] == ["bfloat16"] * 2 + ["float8_e4m3fn"] * 2
    for name, off in found:
        assert 0 <= float(off) <= (2.0 ** -3 if name == "bfloat16" else 2.0 ** -2), text
    norms = re.search(r"gradient norms: q (\S+), k (\S+), v (\S+)", text).groups()
    assert all(0 < float(x) < float("inf") for x in norms)
    assert gdn_lib.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_appended_codes_are_the_definitions(gdn_lib, d):
    """scale = m / 448 with m the largest magnitude of a head's d values, 2^-100 at least, rounded to
    fp32; each code the e4m3 number nearest to 448 x / m in 64 bits, the even one of two."""
    gdn, rows, kv = gdn_lib, 700, 2
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(rows, kv, d, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-120, 100, (rows, kv, 1), generator=g, device="cuda").float())
    x[:40] *= torch.exp2(-20 * torch.rand(40, kv, d, generator=g, device="cuda"))   # small beside the largest
    x[40] = 0
    x[41:60] = torch.randint(-9, 9, (19, kv, d), generator=g, device="cuda").float()  # many ties
    x = x.to(BF16)
    cache = gdn.kv_cache(1, rows, kv, rows, 1, 16, d, FP8)
    ones = torch.ones(rows, dtype=torch.int32, device="cuda")
    gdn.cache_append(cache, x, -x, gdn.cache_reserve(cache, ones))
    values = torch.arange(127, device="cuda", dtype=torch.uint8).view(FP8).double()      # 0 .. 448
    for t, pool, scale in ((x, cache.k, cache.k_scale), (-x, cache.v, cache.v_scale)):
        t = t.double()
        m = t.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
        assert torch.equal(scale[0, :, :, 0], (m[..., 0] / 448).float())
        y = 448 * t / m
        off = (y.abs()[..., None] - values).abs()
        best = off.amin(-1, keepdim=True)
        near = off == best                                  # one, or two beside a tie
        even = near & (torch.arange(127, device="cuda") % 2 == 0)
        code = torch.where(even.any(-1), even.int().argmax(-1), near.int().argmax(-1))
        # (numbers: zero is one, whichever of its two codes stands for it)
        assert torch.equal(pool[0, :, :, 0].double(), values[code] * t.sign())
    assert gdn.device_status() == 0
