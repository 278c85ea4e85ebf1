"""Each direct call (_layer_calls) answers ordinary arguments itself, with one
of the library's launches at least, and gives the general path's bits."""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def rand(*shape, dtype=BF16):
    g = torch.Generator(device=DEV).manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def cases(io):
    """name -> (the direct call's arguments, the public call)."""
    x, r, w = rand(5, 256, dtype=io), rand(5, 256, dtype=io), rand(256, dtype=F32)
    b, wn, wu = rand(5, 256), rand(96, 256), rand(96, 256) + 1
    q, sc = gdn.quantize_fp8(b)
    qw, sw = gdn.quantize_fp8(wn, block_rows=128)
    dh = rand(5, 96)
    code = gdn.GDN_BF16 if io == BF16 else gdn.GDN_F32
    return {
        "residual_norm": ((x, w, r, 1e-5), lambda: gdn.residual_norm(x, w, r)),
        "residual_norm_fp8": ((x, w, r, 1e-5), lambda: gdn.residual_norm_fp8(x, w, r)),
        "residual_norm_backward": ((x, r, w, x, 1e-5),
                                   lambda: gdn.residual_norm_backward(x, r, w, x).values()),
        "quantize_fp8": ((x, 128), lambda: gdn.quantize_fp8(x, 128)),
        "linear_fp8": ((q, sc, qw, sw, code), lambda: gdn.linear_fp8(q, sc, qw, sw, io)),
        "gated_ffn": ((b, wn, wu, gdn.GATE_ACT["sigmoid"]),
                      lambda: gdn.gated_ffn(b, wn, wu, "sigmoid")),
        "gated_ffn_backward": ((b, wn, wu, dh, gdn.GATE_ACT["silu"]),
                               lambda: gdn.gated_ffn_backward(b, wn, wu, dh).values()),
    }


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("name", ["residual_norm", "residual_norm_fp8", "residual_norm_backward",
                                  "quantize_fp8", "linear_fp8", "gated_ffn",
                                  "gated_ffn_backward"])
def test_the_direct_call_answers(io, name, monkeypatch):
    gdn.load()
    args, public = cases(io)[name]
    before = gdn.kernel_launches()
    got = getattr(gdn._direct, name)(*args)
    assert got is not None
    assert gdn.kernel_launches() > before
    monkeypatch.setattr(gdn, "_direct", gdn._Declines())
    want = public()
    as_list = lambda v: [v] if isinstance(v, torch.Tensor) else list(v)  # noqa: E731
    got, want = as_list(got), as_list(want)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and a.shape == b.shape
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
