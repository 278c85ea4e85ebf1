"""Values of the layer operators where fp32 arithmetic loses what the result
still shows: the gate's slope far out.

Tolerances, from the arithmetic.  A one-hot row of x makes G, U and every
product behind them exact, so a weight gradient is the rounding of dG or dU to
bf16, off by 2^-8 of it at most, of a value that is off by the exponential's
argument (|G| 2^-24, twice: the product and its constant), its result (2^-22),
the reciprocal (2^-23) and a few products: below 2^-16 for |G| <= 20.
"""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("tokens,hidden", [(1, 200), (40, 200), (300, 200), (300, 201)])
def test_gate_slope_far_out(act, tokens, hidden):
    dim = (tokens + 7) // 8 * 8
    g = gen(tokens + hidden)
    x = torch.zeros(tokens, dim, dtype=BF16, device=DEV)
    x[torch.arange(tokens), torch.arange(tokens)] = 1
    # G = w_gate transposed: 2..20 either way (SiLU's slope has its root at -1.28)
    wg = (2 + 18 * torch.rand(hidden, dim, generator=g, device=DEV))
    wg = (wg * torch.where(torch.rand(hidden, dim, generator=g, device=DEV) < 0.5, -1.0, 1.0)).to(BF16)
    wu = torch.randn(hidden, dim, generator=g, device=DEV).to(BF16)
    dh = torch.randn(tokens, hidden, generator=g, device=DEV).to(BF16)
    r = gdn.gated_ffn_backward(x, wg, wu, dh, act)
    G, U, d = wg[:, :tokens].double(), wu[:, :tokens].double(), dh.t().double()
    s, c = torch.sigmoid(G), torch.sigmoid(-G)
    a, slope = (G * s, s * (1 + G * c)) if act == "silu" else (s, s * c)
    for name, want in (("dw_gate", d * U * slope), ("dw_up", d * a)):
        off = (r[name][:, :tokens].double() - want).abs() - (2.0 ** -8 + 2.0 ** -16) * want.abs()
        assert float(off.max()) <= 0, (name, float((off / want.abs()).max()))
    assert gdn.device_status() == 0
