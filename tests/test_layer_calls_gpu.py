"""The layer operators' direct calls (_layer_calls) and the binding's general
path give the same bits, and the direct calls decline what is out of the
ordinary instead of answering it."""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def rand(*shape, dtype=BF16):
    g = torch.Generator(device=DEV).manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


@pytest.fixture(params=["direct", "general"])
def path(request, monkeypatch):
    gdn.load()
    assert gdn._direct.__name__.endswith("_layer_calls")   # built, not declining
    if request.param == "general":
        monkeypatch.setattr(gdn, "_direct", gdn._Declines())
    return request.param


def calls(lead=(2, 5)):
    """Every operator's results on fixed inputs."""
    x, r, w = rand(*lead, 256), rand(*lead, 256), rand(256, dtype=torch.float32)
    wn = rand(96, 256)
    out = list(gdn.residual_norm(x, w, r)) + list(gdn.residual_norm(x, w))
    q, sc, s = gdn.residual_norm_fp8(x, w, r, eps=0)
    qw, sw = gdn.quantize_fp8(wn, block_rows=128)
    out += [q, sc, s, qw, sw, *gdn.quantize_fp8(x), *gdn.residual_norm_fp8(x, w)[:2]]
    out += [gdn.linear_fp8(q, sc, qw, sw), gdn.linear_fp8(q, sc, qw, sw, torch.float32)]
    out += gdn.residual_norm_backward(x, s, w, r).values()
    out += gdn.residual_norm_backward(x, s, w).values()
    h = gdn.gated_ffn(x, wn, wn + 1, "sigmoid")
    out += [h, *gdn.gated_ffn_backward(x, wn, wn + 1, h, "silu").values()]
    return out


def test_both_paths_agree(path, monkeypatch):
    got = calls()
    monkeypatch.undo()
    want = calls()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(
            a.view(torch.uint8), b.view(torch.uint8))


def test_sum_without_residual_is_x(path):
    x, w = rand(4, 64), rand(64, dtype=torch.float32)
    assert gdn.residual_norm(x, w)[1] is x and gdn.residual_norm_fp8(x, w)[2] is x


def test_direct_calls_decline():
    gdn.load()
    d = gdn._direct
    x, w, wn = rand(4, 64), rand(64, dtype=torch.float32), rand(32, 64)
    q, sc = gdn.quantize_fp8(x)
    qw, sw = gdn.quantize_fp8(wn, block_rows=128)
    before = gdn.kernel_launches()
    assert d.residual_norm(x.cpu(), w, None, 1e-5) is None
    assert d.residual_norm(x.t(), w, None, 1e-5) is None             # strides
    assert d.residual_norm(x.half(), w, None, 1e-5) is None
    assert d.residual_norm(x, w, x[:2], 1e-5) is None
    assert d.residual_norm(x, w, None, "small") is None
    assert d.residual_norm(x, w, None, -1.0) is None                 # the library's refusal
    assert d.residual_norm(x[:, :60].contiguous(), w[:60].contiguous(), None, 1e-5) is None
    assert d.residual_norm(x[:0], w, None, 1e-5) is None
    assert d.residual_norm_fp8(x, x[0], None, 1e-5) is None
    assert d.residual_norm_backward(x[:2], x, w, None, 1e-5) is None
    assert d.quantize_fp8(x, 64) is None and d.quantize_fp8(x, None) is None
    assert d.linear_fp8(q, sc, qw, sw, 7) is None
    assert d.linear_fp8(q, sc[:2], qw, sw, 1) is None
    assert d.linear_fp8(x, sc, qw, sw, 1) is None
    assert d.gated_ffn(x, wn, wn[:8], 0) is None and d.gated_ffn(x, wn, wn, None) is None
    assert d.gated_ffn_backward(x, wn, wn, x, 0) is None
    assert gdn.kernel_launches() == before
    with pytest.raises(gdn.GDNError):
        gdn.residual_norm(x, w, eps=-1.0)
    with pytest.raises(TypeError):
        gdn.residual_norm(x.half(), w)
    with pytest.raises(ValueError):
        gdn.gated_ffn(x, wn, wn, act="tanh")


def test_other_streams(path):
    x, w = rand(300, 256), rand(256, dtype=torch.float32)
    want = gdn.residual_norm(x, w)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gdn.residual_norm(x, w)[0]
    side.synchronize()
    assert torch.equal(got, want)
