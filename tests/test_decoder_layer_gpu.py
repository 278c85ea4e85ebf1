"""The decoder layer of examples/decoder_layer.py: prefill against decoding
from its states, and the training half against differentiating the same
formulas in fp32.

Tolerances: both serving paths round the same quantities to bf16 (2^-8) and to
e4m3 (2^-4) at the same places, but from values that differ by a rounding to
bf16 (q, k and v stay fp32 in the decode step), so a share of the 8-bit codes
differs by a step; the two e4m3 roundings behind the mixer (2^-4 each, at
most) bound the outputs' relative difference by 2^-3.  Gradients: bf16
roundings of z, dG, dU, dz and the results, 2^-8 each, and as many again in
the terms they enter: 2^-5.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
pytestmark = pytest.mark.gpu


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.fixture(scope="module")
def layer():
    from decoder_layer import DecoderLayer
    return DecoderLayer(dim=400, heads=2, hidden=528, seed=3)


def test_decoding_continues_the_prefill(layer):
    import hybrid_linear_attention_deltanet_gb300 as gdn
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(3, 40, layer.dim, generator=g, device="cuda").bfloat16()
    r = torch.randn(3, 40, layer.dim, generator=g, device="cuda").bfloat16()
    whole, stream, _ = layer.prefill(x, r)
    _, _, state = layer.prefill(x[:, :33].contiguous(), r[:, :33].contiguous())
    for t in range(33, 40):
        out, res = layer.decode(x[:, t].contiguous(), state, r[:, t].contiguous())
        assert rel(out, whole[:, t]) <= 2.0 ** -3
        assert rel(res, stream[:, t]) <= 2.0 ** -3
    assert gdn.device_status() == 0


def test_training_half(layer):
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    o, res, dh, dres = rand(90, 400), rand(90, 400), rand(90, 528), rand(90, 400)
    got = layer.train_feed_forward(o, res, dh, dres)
    s = (o.float() + res.float()).bfloat16().double().requires_grad_()
    w = [t.double().requires_grad_() for t in (layer.norm2, layer.w_gate, layer.w_up)]
    z = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-5) * w[0]
    h = torch.nn.functional.silu(z @ w[1].t()) * (z @ w[2].t())
    ((h * dh.double()).sum() + (s * dres.double()).sum()).backward()
    for a, b in zip(got, [h.detach(), s.grad, *(t.grad for t in w)]):
        assert rel(a, b) <= 2.0 ** -5


def test_example_runs(capsys):
    import decoder_layer
    decoder_layer.main()
    assert "gradient norms" in capsys.readouterr().out
