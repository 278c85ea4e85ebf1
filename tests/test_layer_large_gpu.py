"""Tensors of more than 2^31 elements: every row of a large call, made of
copies of a small one, has the small call's bits (rows do not mix), beyond the
2^31st element too.  Sums over the rows are compared within their roundings."""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    gdn.release_scratch()


def randn(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def same_rows(big, small, copies):
    """Every copy has the small tensor's bits."""
    rows = small.shape[0]
    for i in range(copies):
        if not torch.equal(big[i * rows:(i + 1) * rows].view(torch.uint8), small.view(torch.uint8)):
            return False
    return True


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


ROWS, DIM, COPIES = 8192, 8192, 33          # 33 x 2^26 elements


def test_norms():
    x, r, w = randn(1, ROWS, DIM), randn(2, ROWS, DIM), 1 + randn(3, DIM, dtype=F32, scale=0.1)
    y, s = gdn.residual_norm(x, w, r)
    q, scale, _ = gdn.residual_norm_fp8(x, w, r)
    X, R = x.repeat(COPIES, 1), r.repeat(COPIES, 1)
    assert X.numel() > 2 ** 31
    Q, SC, S = gdn.residual_norm_fp8(X, w, R)
    assert same_rows(Q, q, COPIES) and same_rows(SC, scale, COPIES) and same_rows(S, s, COPIES)
    del Q, SC, S
    gdn.residual_norm(X, w, R, s=R, y=X)
    assert same_rows(X, y, COPIES) and same_rows(R, s, COPIES)


def test_norm_gradient():
    s, dy, w = randn(4, ROWS, DIM), randn(5, ROWS, DIM), 1 + randn(6, DIM, dtype=F32, scale=0.1)
    a = gdn.residual_norm_backward(dy, s, w, s)
    S = s.repeat(COPIES, 1)
    b = gdn.residual_norm_backward(dy.repeat(COPIES, 1), S, w, S)
    assert same_rows(b["dx"], a["dx"], COPIES)
    # fp32 sums in another order: about sqrt(rows) 2^-24
    assert rel(b["dw"], COPIES * a["dw"].double()) <= 2.0 ** -14


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantisation(block_rows):
    x = randn(7, ROWS, DIM)
    q, scale = gdn.quantize_fp8(x, block_rows)
    Q, SC = gdn.quantize_fp8(x.repeat(COPIES, 1), block_rows)
    assert Q.numel() > 2 ** 31
    assert same_rows(Q, q, COPIES) and same_rows(SC, scale, COPIES)


@pytest.mark.parametrize("n", [2005, 2008])
def test_product(n):
    tokens, k, copies = 8192, 144, 132
    x, sx = gdn.quantize_fp8(randn(8, tokens, k))
    w, sw = gdn.quantize_fp8(randn(9, n, k), block_rows=128)
    out = gdn.linear_fp8(x, sx, w, sw)
    big = gdn.linear_fp8(x.view(torch.uint8).repeat(copies, 1).view(gdn.FP8), sx.repeat(copies, 1),
                         w, sw)
    assert big.numel() > 2 ** 31
    assert same_rows(big, out, copies)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("hidden", [8000, 8001])
def test_feed_forward(hidden):
    tokens, dim, copies = 2048, 64, 132
    x, dh = randn(10, tokens, dim), randn(11, tokens, hidden, scale=0.1)
    wg, wu = (randn(s, hidden, dim, scale=dim ** -0.5) for s in (12, 13))
    h, a = gdn.gated_ffn(x, wg, wu), gdn.gated_ffn_backward(x, wg, wu, dh)
    X = x.repeat(copies, 1)
    H = gdn.gated_ffn(X, wg, wu)
    assert H.numel() > 2 ** 31
    assert same_rows(H, h, copies)
    del H
    b = gdn.gated_ffn_backward(X, wg, wu, dh.repeat(copies, 1))
    # the same dG and dU in fp32 sums of another order, both results rounded to
    # bf16 (2^-8 at most, in norm half of it each)
    assert rel(b["dx"], a["dx"].repeat(copies, 1)) <= 2.0 ** -8
    for name in ("dw_gate", "dw_up"):
        assert rel(b[name], copies * a[name].double()) <= 2.0 ** -8
    assert gdn.device_status() == 0
