"""Calls of the layer operators queued one behind the other without a
synchronisation, with other inputs each time and on the same memory, give what
each gives alone: grids of one call may be resident while those of the call
before still run."""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def randn(g, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def alone(f, sets):
    """Each set's results with nothing else in flight."""
    out = []
    for s in sets:
        torch.cuda.synchronize()
        out.append([t.clone() for t in f(s)])
        torch.cuda.synchronize()
    return out


def check_queue(f, sets, rounds=40):
    want = alone(f, sets)
    order = [(3 * i + i // 7) % len(sets) for i in range(rounds)]
    got = [[t.clone() for t in f(sets[i])] for i in order]
    torch.cuda.synchronize()
    for i, r in zip(order, got):
        for a, b in zip(r, want[i]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert gdn.device_status() == 0


# dx in parts; the weight gradients in parts; neither, many tokens; rows of dh
# that start anywhere
@pytest.mark.parametrize("tokens,dim,hidden", [(32, 256, 2048), (1111, 264, 2731), (300, 72, 700),
                                               (260, 520, 1001)])
def test_feed_forward_gradients(tokens, dim, hidden):
    sets = []
    for i in range(4):
        g = gen(100 * tokens + i)
        sets.append([randn(g, tokens, dim), randn(g, hidden, dim, scale=dim ** -0.5),
                     randn(g, hidden, dim, scale=dim ** -0.5), randn(g, tokens, hidden)])
    ws = torch.empty(gdn.gated_ffn_backward_workspace_size(tokens, dim, hidden),
                     dtype=torch.uint8, device=DEV)
    check_queue(lambda s: list(gdn.gated_ffn_backward(*s, workspace=ws).values()), sets)
    check_queue(lambda s: list(gdn.gated_ffn_backward(*s).values()), sets)


@pytest.mark.parametrize("tokens,dim", [(300, 256), (1300, 4096), (5000, 1024)])
def test_norm_gradient(tokens, dim):
    sets = []
    for i in range(4):
        g = gen(tokens + i)
        sets.append([randn(g, tokens, dim), randn(g, tokens, dim), randn(g, dim, dtype=F32)])
    ws = torch.empty(max(1, gdn.residual_norm_backward_workspace_size(tokens, dim)),
                     dtype=torch.uint8, device=DEV)
    check_queue(lambda s: list(gdn.residual_norm_backward(*s, workspace=ws).values()), sets)


@pytest.mark.parametrize("tokens", [1, 40, 300, 1500])
def test_products_of_buffers_written_just_before(tokens):
    """Codes, scales, sums and dh live in buffers that the call before writes."""
    dim, n, hidden = 640, 520, 264
    g = gen(tokens)
    wq = gdn.quantize_fp8(randn(g, n, dim, scale=dim ** -0.5), block_rows=128)
    w = 1 + 0.1 * randn(g, dim, dtype=F32)
    wh = 1 + 0.1 * randn(g, hidden, dtype=F32)
    wg, wu = randn(g, hidden, dim, scale=dim ** -0.5), randn(g, hidden, dim, scale=dim ** -0.5)
    q = torch.empty(tokens, dim, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(tokens, dim // 128, device=DEV)
    y = torch.empty(tokens, dim, dtype=BF16, device=DEV)
    dh = torch.empty(tokens, hidden, dtype=BF16, device=DEV)

    def layer(s):
        x, r, h = s
        gdn.residual_norm_fp8(x, w, q=q, scale=scale)
        out = gdn.linear_fp8(q, scale, *wq)
        gdn.residual_norm(r, w, y=y)
        gdn.residual_norm(h, wh, y=dh)
        return [out, *gdn.gated_ffn_backward(y, wg, wu, dh).values()]

    sets = []
    for i in range(4):
        # blocks of 128 columns louder and quieter than their row, so that scales differ
        loud = torch.exp2(
            torch.randint(-3, 4, (tokens, dim // 128, 1), generator=g, device=DEV).float())
        x = randn(g, tokens, dim // 128, 128, dtype=F32) * loud
        sets.append([x.view(tokens, dim).to(BF16), randn(g, tokens, dim),
                     randn(g, tokens, hidden)])
    check_queue(layer, sets)
