"""The operators around the mixer refuse malformed host arguments before they
touch the GPU, at the C ABI (status codes) and in the Python binding.  CPU
only: the C calls get fake addresses and do not run where a CUDA device is
visible, so a missed check can never reach a GPU."""
import ctypes

import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn
from test_abi import fake_addresses, lib  # noqa: F401  (fixture)

P = ctypes.c_void_p
SIZE_MAX = ctypes.c_size_t(-1).value
X, R, W, S, Y, Q, SC = (P(0x1000000 * (i + 1)) for i in range(7))
MIS = P(0x1000008)
BF16, F32 = 1, 0


@pytest.fixture(autouse=True)
def no_launch(request):
    if "lib" not in request.fixturenames:
        yield
        return
    library = request.getfixturevalue("lib")
    before = library.gdn_kernel_launches()
    yield
    assert library.gdn_kernel_launches() == before, "a host-argument test launched a kernel"


@fake_addresses
def test_residual_norm_refuses(lib):  # noqa: F811
    def f(x=X, r=R, w=W, eps=1e-5, s=S, y=Y, t=16, d=256, io=BF16):
        return lib.gdn_residual_norm(x, r, w, eps, s, y, t, d, io, None)
    assert f(t=0) == 0
    assert f(t=-1) == 1 and f(d=0) == 1 and f(eps=-1.0) == 1 and f(eps=float("nan")) == 1
    assert f(x=None) == 1 and f(w=None) == 1 and f(y=None) == 1
    assert f(s=None) == 1 and f(r=None) == 1          # residual and s go together
    assert f(d=260) == 2 and f(d=16392) == 2 and f(io=2) == 2
    assert f(x=MIS) == 3 and f(y=P(0x5000004)) == 3 and f(w=P(0x3000004)) == 3
    assert f(y=S) == 1                                # two outputs in one place
    assert f(y=P(0x1000000 + 512)) == 1               # y inside x, not x itself
    assert f(s=P(0x2000000 + 512)) == 1 and f(s=W) == 1


@fake_addresses
def test_residual_norm_fp8_refuses(lib):  # noqa: F811
    def f(x=X, r=R, w=W, eps=1e-5, s=S, q=Q, sc=SC, t=16, d=256, io=BF16):
        return lib.gdn_residual_norm_fp8(x, r, w, eps, s, q, sc, t, d, io, None)
    assert f(t=0) == 0
    assert f(q=None) == 1 and f(sc=None) == 1 and f(x=None) == 1
    assert f(d=12) == 2 and f(io=9) == 2
    assert f(q=P(0x6000008)) == 3 and f(sc=P(0x7000002)) == 3
    assert f(q=X) == 1 and f(q=S) == 1 and f(sc=Q) == 1 and f(sc=P(0x3000010)) == 1


@fake_addresses
def test_residual_norm_backward_refuses(lib):  # noqa: F811
    dw = SC

    def f(dy=X, s=R, w=W, ds=None, eps=1e-5, dx=Y, dw=dw, t=16, d=256, io=BF16):
        return lib.gdn_residual_norm_backward(dy, s, w, ds, eps, dx, dw, t, d, io, None)
    assert f(dy=None) == 1 and f(s=None) == 1 and f(dx=None) == 1 and f(dw=None) == 1
    assert f(w=None) == 1 and f(t=-1) == 1 and f(eps=-1.0) == 1
    assert f(d=12) == 2 and f(io=4) == 2
    assert f(dy=MIS) == 3 and f(dw=P(0x7000008)) == 3
    assert f(dx=X) == 1 and f(dw=W) == 1 and f(dx=P(0x2000000 + 16)) == 1
    size = lib.gdn_residual_norm_backward_workspace_size
    assert size(300, 256, BF16) == 19 * 256 * 4 and size(256, 256, BF16) == 0
    assert size(0, 256, BF16) == 0
    assert size(1 << 20, 4096, BF16) == 608 * 4096 * 4
    assert size(16, 12, BF16) == SIZE_MAX and size(-1, 256, BF16) == SIZE_MAX
    ws = P(0x9000000)

    def g(ws=ws, n=19 * 256 * 4):
        return lib.gdn_residual_norm_backward_ws(X, R, W, None, 1e-5, Y, dw, 300, 256, BF16, ws, n,
                                                 None)
    assert g(ws=None) == 1 and g(n=19 * 256 * 4 - 1) == 1 and g(ws=P(0x9000010)) == 3 and g(ws=X) == 1


@fake_addresses
def test_quantize_fp8_refuses(lib):  # noqa: F811
    def f(x=X, q=Q, sc=SC, rows=16, cols=256, br=1, io=BF16):
        return lib.gdn_quantize_fp8(x, q, sc, rows, cols, br, io, None)
    assert f(rows=0) == 0
    assert f(rows=-1) == 1 and f(cols=0) == 1 and f(x=None) == 1 and f(q=None) == 1
    assert f(cols=20) == 2 and f(br=64) == 2 and f(io=5) == 2
    assert f(x=MIS) == 3 and f(sc=P(0x7000001)) == 3
    assert f(q=X) == 1 and f(sc=Q) == 1


@fake_addresses
def test_linear_fp8_refuses(lib):  # noqa: F811
    def f(x=X, sx=R, w=W, sw=S, out=Y, t=16, k=256, n=128, dt=BF16):
        return lib.gdn_linear_fp8(x, sx, w, sw, out, t, k, n, dt, None)
    assert f(t=0) == 0
    assert f(t=-1) == 1 and f(k=0) == 1 and f(n=0) == 1
    assert f(x=None) == 1 and f(sx=None) == 1 and f(w=None) == 1 and f(sw=None) == 1
    assert f(out=None) == 1
    assert f(k=264) == 2 and f(dt=3) == 2 and f(t=1 << 31) == 2
    assert f(x=MIS) == 3 and f(w=P(0x3000004)) == 3 and f(out=P(0x5000002)) == 3
    assert f(sx=P(0x2000002)) == 3
    assert f(out=X) == 1 and f(out=P(0x3000010)) == 1


@fake_addresses
def test_gated_ffn_refuses(lib):  # noqa: F811
    def f(x=X, wg=R, wu=W, act=0, h=Y, t=16, d=256, hid=512, io=BF16):
        return lib.gdn_gated_ffn(x, wg, wu, act, h, t, d, hid, io, None)
    assert f(t=0) == 0
    assert f(t=-1) == 1 and f(d=0) == 1 and f(hid=0) == 1
    assert f(x=None) == 1 and f(wg=None) == 1 and f(wu=None) == 1 and f(h=None) == 1
    assert f(d=260) == 2 and f(act=2) == 2 and f(io=F32) == 2 and f(t=1 << 31) == 2
    assert f(x=MIS) == 3 and f(h=P(0x5000008)) == 3
    assert f(h=X) == 1 and f(h=P(0x3000010)) == 1


@fake_addresses
def test_gated_ffn_backward_refuses(lib):  # noqa: F811
    def f(x=X, wg=R, wu=W, dh=S, act=0, dx=Y, dwg=Q, dwu=SC, t=16, d=256, hid=512, io=BF16):
        return lib.gdn_gated_ffn_backward(x, wg, wu, dh, act, dx, dwg, dwu, t, d, hid, io, None)
    assert f(t=-1) == 1 and f(dh=None) == 1 and f(dx=None) == 1 and f(dwg=None) == 1
    assert f(dwu=None) == 1 and f(wg=None) == 1
    assert f(d=12) == 2 and f(act=-1) == 2 and f(io=F32) == 2
    assert f(dh=P(0x4000004)) == 3 and f(dwu=P(0x7000008)) == 3
    assert f(dx=X) == 1 and f(dwg=SC) == 1 and f(dwu=R) == 1
    size = lib.gdn_gated_ffn_backward_workspace_size
    assert size(16, 256, 512, BF16) == 2 * 16 * 512 * 2 and size(0, 256, 512, BF16) == 0
    assert size(3, 256, 17, BF16) == 2 * 256          # rows on 32 bytes, arrays on 256
    assert size(16, 256, 512, F32) == SIZE_MAX and size(16, 12, 512, BF16) == SIZE_MAX
    n = size(16, 256, 512, BF16)

    def g(ws=P(0x9000000), n=n):
        return lib.gdn_gated_ffn_backward_ws(X, R, W, S, 0, Y, Q, SC, 16, 256, 512, BF16, ws, n,
                                             None)
    assert g(ws=None) == 1 and g(n=n - 1) == 1 and g(ws=P(0x9000080)) == 3 and g(ws=S) == 1


# ---------------------------------------------------- the binding's own checks
def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_shapes_types_and_strides(lib):  # noqa: F811
    w = t(64, dtype=torch.float32)
    with pytest.raises(ValueError):
        gdn.residual_norm(t(4, 64), t(32, dtype=torch.float32))
    with pytest.raises(TypeError):
        gdn.residual_norm(t(4, 64), t(64))                        # w is fp32
    with pytest.raises(TypeError):
        gdn.residual_norm(t(4, 64, dtype=torch.float16), w)
    with pytest.raises(ValueError):
        gdn.residual_norm(t(64, 4).t(), t(64, dtype=torch.float32))
    with pytest.raises(ValueError):
        gdn.residual_norm(t(4, 64), w, residual=t(3, 64))
    with pytest.raises(ValueError):
        gdn.residual_norm(t(4, 64), w, s=t(4, 64))                # s without a residual
    with pytest.raises(ValueError):
        gdn.residual_norm_fp8(t(4, 64), w, scale=t(4, 2, dtype=torch.float32))
    with pytest.raises(ValueError):
        gdn.residual_norm_backward(t(4, 64), t(5, 64), w)
    with pytest.raises(TypeError):
        gdn.residual_norm_backward(None, t(5, 64), w)
    with pytest.raises(ValueError):
        gdn.quantize_fp8(t(4, 64), block_rows=64)
    with pytest.raises(ValueError):
        gdn.quantize_fp8(t(2, 4, 64), block_rows=128)
    f8 = lambda *s: torch.zeros(*s, dtype=torch.uint8).view(gdn.FP8)  # noqa: E731
    f32 = lambda *s: t(*s, dtype=torch.float32)  # noqa: E731
    with pytest.raises(TypeError):
        gdn.linear_fp8(t(4, 256), f32(4, 2), f8(8, 256), f32(1, 2))
    with pytest.raises(ValueError):
        gdn.linear_fp8(f8(4, 256), f32(4, 3), f8(8, 256), f32(1, 2))
    with pytest.raises(ValueError):
        gdn.linear_fp8(f8(4, 256), f32(4, 2), f8(8, 256), f32(2, 2))
    with pytest.raises(ValueError):
        gdn.linear_fp8(f8(4, 256), f32(4, 2), f8(8, 128), f32(1, 1))
    with pytest.raises(TypeError):
        gdn.linear_fp8(f8(4, 256), f32(4, 2), f8(8, 256), f32(1, 2), torch.float16)
    with pytest.raises(TypeError):
        gdn.gated_ffn(f32(4, 64), f32(8, 64), f32(8, 64))
    with pytest.raises(ValueError):
        gdn.gated_ffn(t(4, 64), t(8, 64), t(9, 64))
    with pytest.raises(ValueError):
        gdn.gated_ffn(t(4, 64), t(8, 64), t(8, 64), act="gelu")
    with pytest.raises(ValueError):
        gdn.gated_ffn(t(4, 64), t(8, 64), t(8, 64), h=t(4, 9))
    with pytest.raises(ValueError):
        gdn.gated_ffn_backward(t(4, 64), t(8, 64), t(8, 64), t(4, 9))
    with pytest.raises(ValueError):
        gdn.gated_ffn_backward_workspace_size(4, 12, 8)
    with pytest.raises(ValueError):
        gdn.residual_norm_backward_workspace_size(4, 12)
