"""Values of the layer operators where fp32 arithmetic loses what the result
still shows: the gate's slope far out, and 8-bit codes on and beside the middle
between two codes below e4m3's normal range and near fp32's largest numbers.

Tolerances, from the arithmetic.  A one-hot row of x makes G, U and every
product behind them exact, so a weight gradient is the rounding of dG or dU to
bf16, off by 2^-8 of it at most, of a value that is off by the exponential's
argument (|G| 2^-24, twice: the product and its constant), its result (2^-22),
the reciprocal (2^-23) and a few products: below 2^-16 for |G| <= 20.  Codes
are compared exactly.
"""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


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


def e4m3_of(v):
    """e4m3 value nearest to v (64 bits, |v| <= 448), ties to even: 3 fraction bits, exponents
    from -6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def middles(g, shape):
    """Random middles between two e4m3 codes, half of them below the normal range."""
    odd = 2 * torch.randint(0, 8, shape, generator=g, device=DEV) + 1
    low = odd.double() * 2.0 ** -10
    e = torch.randint(-6, 8, shape, generator=g, device=DEV).double()
    high = (16 + odd.double()) * torch.exp2(e - 4)
    high = high.clamp_max(440.0)   # 448 is the last code
    v = torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, low, high)
    return v * torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, -1.0, 1.0)


def check_codes_about_middles(io, block_rows, exponent):
    """x = c t 2^e, for fp32 and its neighbours too, in blocks whose maximum is
    448 c 2^e: 448 x / m is the middle t, or just beside it."""
    g = gen(exponent + block_rows + 200)
    rows, cols = 512, 1024
    c = torch.randint(1, 4096 if io == F32 else 8, (rows // block_rows, 1, cols // 128, 1),
                      generator=g, device=DEV)
    t = middles(g, (rows // block_rows, block_rows, cols // 128, 128))
    x = (c.double() * t * 2.0 ** exponent).to(io)
    if io == F32:
        way = torch.randint(-1, 2, x.shape, generator=g, device=DEV)
        to = torch.where(way > 0, 3.4e38, -3.4e38).to(io)
        x = torch.where(way == 0, x, torch.nextafter(x, to))
    x[:, 0, :, 0] = (448 * c.double() * 2.0 ** exponent).to(io)[:, 0, :, 0]
    x = x.view(rows, cols).contiguous()
    assert bool(torch.isfinite(x).all())
    q, scale = gdn.quantize_fp8(x, block_rows=block_rows)
    b = x.double().view(rows // block_rows, block_rows, cols // 128, 128)
    want = e4m3_of(448 * b / b.abs().amax((1, 3), keepdim=True)).view(rows, cols)
    assert torch.equal(q.double(), want)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("exponent", [0, -100])
def test_quantised_codes_on_and_beside_the_middles(io, block_rows, exponent):
    check_codes_about_middles(io, block_rows, exponent)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantised_codes_near_the_largest_numbers(block_rows):
    """448 x passes fp32's largest number here: block maxima to 1.8e6 2^107."""
    check_codes_about_middles(F32, block_rows, 107)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantised_codes_below_the_least_maximum(block_rows):
    """Blocks whose maximum is below 2^-100 take that in its place: 448 x 2^100 is
    beside a middle (7 divides no power of two)."""
    g = gen(block_rows + 300)
    x = (middles(g, (512, 1024)) * 2.0 ** -106 / 7).float()
    way = torch.randint(-1, 2, x.shape, generator=g, device=DEV)
    x = torch.where(way == 0, x, torch.nextafter(x, torch.where(way > 0, 1.0, -1.0)))
    q, scale = gdn.quantize_fp8(x, block_rows=block_rows)
    assert bool((scale == torch.tensor(2.0 ** -100, device=DEV) / 448).all())
    assert torch.equal(q.double(), e4m3_of(448 * x.double() * 2.0 ** 100))


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("rows", [2048, 300, 1])
def test_norm_codes_below_the_normal_range(io, rows):
    """The norm's root cancels in 448 y / max |y|: s and w with few bits put many
    values on the middles below the normal range."""
    g = gen(rows + 7)
    x = torch.randint(-40, 41, (rows, 1024), generator=g, device=DEV).to(io) * 2.0 ** -10
    loud = torch.randint(1, 4, (rows, 8), generator=g, device=DEV)
    x[:, ::128] = (448 * loud).to(io)
    w = torch.randint(1, 9, (1024,), generator=g, device=DEV).float() / 4
    w[::128] = 1.0
    q, _, _ = gdn.residual_norm_fp8(x, w)
    p = (x.double() * w.double()).view(rows, 8, 128)
    want = e4m3_of((448 * p / p.abs().amax(-1, keepdim=True)).view(rows, 1024))
    assert torch.equal(q.double(), want)
