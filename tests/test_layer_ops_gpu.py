"""GPU tests of the operators around the mixer (gdn_residual_norm and its
8-bit and gradient forms, gdn_quantize_fp8, gdn_linear_fp8, gdn_gated_ffn and
its gradient) against their formulas in 64 bits.

Tolerances, from the arithmetic.  Rounding to bf16 is off by at most 2^-8 of
the value, to e4m3 by 2^-4 (or half its smallest step, 2^-10, times the
scale), to fp32 by 2^-24.  A tensor-core product of K bf16 terms adds 16 of
them at a time to an fp32 accumulator, each addition off by at most 2^-23 of
the largest partial sum, which S = sum |a b| bounds: (K / 16 + 1) 2^-23 S.
For 8-bit operands the width of the inner accumulator is not documented; with
13 bits or more below the largest term it is off by at most 2^-13 S.  The
activation's exponential and reciprocal are each good to 2^-21.
"""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
EPS = 1e-5


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def frob(a, b):
    d = (a.double() - b.double()).norm()
    n = b.double().norm()
    return float(d / n) if n > 0 else float(d)


def within(a, ref, bound, what=""):
    """Elementwise |a - ref| <= bound."""
    over = (a.double() - ref).abs() - bound
    assert not torch.isnan(over).any(), what
    assert float(over.max()) <= 0 if over.numel() else True, (what, float(over.max()))


class Guarded:
    """An output inside a larger buffer whose surroundings must stay as they were."""

    def __init__(self, shape, dtype, pad=256):
        n = int(np.prod(shape))
        item = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full(((n + 2 * pad) * item,), 0x5A, dtype=torch.uint8, device=DEV)
        self.lo, self.hi = pad * item, (pad + n) * item
        self.t = self.raw[self.lo:self.hi].view(dtype).view(shape)

    def check(self):
        assert bool((self.raw[:self.lo] == 0x5A).all()) and bool((self.raw[self.hi:] == 0x5A).all())


# -------------------------------------------------------------------- norm
def norm_ref(x, r, w, io):
    s = x if r is None else (x.float() + r.float()).to(io)
    d = s.double()
    rs = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    return s, d * rs * w.double()


NORM_DIMS = [8, 72, 128, 256, 264, 520, 1032, 2048, 2056, 4096, 8192, 16384]


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("res", [True, False])
def test_residual_norm(io, dim, res):
    g = gen(dim)
    for tokens in (1, 9, 67):
        x, w = randn(g, tokens, dim, dtype=io), 1 + 0.1 * randn(g, dim)
        r = randn(g, tokens, dim, dtype=io) if res else None
        yb, sb = Guarded((tokens, dim), io), Guarded((tokens, dim), io)
        y, s = gdn.residual_norm(x, w, r, EPS, s=sb.t if res else None, y=yb.t)
        s_ref, y_ref = norm_ref(x, r, w, io)
        assert torch.equal(s, s_ref)
        # the sum of squares, its root and three products in fp32
        within(y, y_ref, (HALF[io] + dim * 2.0 ** -24 + 2.0 ** -20) * y_ref.abs(), "y")
        yb.check(), sb.check()
        if not res:
            assert s.data_ptr() == x.data_ptr()
    assert gdn.device_status() == 0


def block_view(t, blocks):
    out = torch.zeros(t.shape[0], blocks * 128, dtype=torch.float64, device=t.device)
    out[:, :t.shape[1]] = t.double()
    return out.view(t.shape[0], blocks, 128)


def check_quantised(q, scale, ref, rel):
    """q * scale against the fp64 values `ref`, themselves known to `rel` in fp32."""
    blocks = -(-ref.shape[1] // 128)
    assert scale.shape == (ref.shape[0], blocks)
    b = block_view(ref, blocks)
    m = b.abs().amax(-1).clamp_min(2.0 ** -100)
    within(scale, m / 448, (rel + 2.0 ** -23) * m / 448, "scale")
    got = block_view(q.float(), blocks) * scale.double()[..., None]
    within(got, b, (2.0 ** -4 + 2 * rel) * b.abs() + 2.0 ** -10 * (m / 448)[..., None] * (1 + rel),
           "q")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("dim", NORM_DIMS)
def test_residual_norm_fp8(io, dim):
    g = gen(dim + 1)
    for tokens in (1, 9, 67):
        x, w, r = randn(g, tokens, dim, dtype=io), 1 + 0.1 * randn(g, dim), randn(g, tokens, dim, dtype=io)
        x[:, ::31] *= 20
        qb, sb = Guarded((tokens, dim), FP8), Guarded((tokens, -(-dim // 128)), F32)
        q, scale, s = gdn.residual_norm_fp8(x, w, r, EPS, q=qb.t, scale=sb.t)
        s_ref, y_ref = norm_ref(x, r, w, io)
        assert torch.equal(s, s_ref)
        check_quantised(q, scale, y_ref, dim * 2.0 ** -24 + 2.0 ** -20)
        # the block's largest value is held exactly as 448 scale
        top = block_view(q.float(), scale.shape[1]).abs().amax(-1)
        assert bool((top == 448).all())
        qb.check(), sb.check()


def test_norm_in_place_and_zero_rows():
    g = gen(3)
    x, r, w = randn(g, 65, 2056, dtype=BF16), randn(g, 65, 2056, dtype=BF16), 1 + randn(g, 2056)
    y0, s0 = gdn.residual_norm(x, w, r)
    xa, ra = x.clone(), r.clone()
    y, s = gdn.residual_norm(xa, w, ra, s=ra, y=xa)
    assert torch.equal(y, y0) and torch.equal(s, s0) and s.data_ptr() == ra.data_ptr()
    # a row of zeros stays zero, in 8 bits with the smallest scale
    z = torch.zeros(2, 2056, dtype=BF16, device=DEV)
    y, _ = gdn.residual_norm(z, w)
    q, scale, _ = gdn.residual_norm_fp8(z, w)
    assert float(y.abs().max()) == 0 and float(q.float().abs().max()) == 0
    assert torch.all(scale == torch.tensor(2.0 ** -100, device=DEV) / 448)
    # no tokens: nothing happens
    e = torch.zeros(0, 2056, dtype=BF16, device=DEV)
    y, _ = gdn.residual_norm(e, w)
    q, scale, _ = gdn.residual_norm_fp8(e, w)
    assert y.shape == (0, 2056) and q.shape == (0, 2056) and scale.shape == (0, 17)
    b = gdn.residual_norm_backward(e, e, w)
    assert b["dx"].shape == (0, 2056) and float(b["dw"].abs().max()) == 0


def test_quantised_nan_and_infinity_show():
    g = gen(4)
    x = randn(g, 3, 384, dtype=BF16)
    x[0, 5], x[1, 130] = float("nan"), float("inf")
    q, scale = gdn.quantize_fp8(x)
    v = block_view(q.float(), 3) * scale.double()[..., None]
    bad = torch.zeros(3, 3, dtype=torch.bool, device=DEV)
    bad[0, 0] = bad[1, 1] = True
    assert torch.equal(torch.isnan(v).all(-1), bad) and torch.equal(torch.isnan(v).any(-1), bad)
    w = torch.ones(384, device=DEV)
    q, scale, _ = gdn.residual_norm_fp8(x, w)
    v = block_view(q.float(), 3) * scale.double()[..., None]
    assert bool(torch.isnan(v[0]).all()) and not bool(torch.isnan(v[2]).any())
    assert bool(torch.isnan(v[1, 1]).all())


def norm_backward_ref(dy, s, w, ds):
    d, f = dy.double(), s.double()
    rs = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    n, gw = f * rs, d * w.double()
    dx = (gw - n * (gw * n).mean(-1, keepdim=True)) * rs
    return (dx if ds is None else dx + ds.double()), (d * n).sum(0), (gw.abs() + n.abs() * (gw * n).abs().mean(-1, keepdim=True)) * rs, (d * n).abs().sum(0)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("res", [True, False])
def test_residual_norm_backward(io, dim, res):
    g = gen(dim + 2)
    for tokens in (1, 9, 333, 1300):
        s, dy = randn(g, tokens, dim, dtype=io), randn(g, tokens, dim, dtype=io)
        ds, w = (randn(g, tokens, dim, dtype=io) if res else None), 1 + 0.1 * randn(g, dim)
        r = gdn.residual_norm_backward(dy, s, w, ds, EPS)
        dx, dw, mx, mw = norm_backward_ref(dy, s, w, ds)
        acc = dim * 2.0 ** -23 + 2.0 ** -19
        within(r["dx"], dx, (HALF[io] + 2.0 ** -23) * dx.abs() + acc * mx, "dx")
        within(r["dw"], dw, (acc + tokens * 2.0 ** -24) * mw, "dw")
        ws = torch.empty(gdn.residual_norm_backward_workspace_size(tokens, dim, io),
                         dtype=torch.uint8, device=DEV)
        again = gdn.residual_norm_backward(dy, s, w, ds, EPS, workspace=ws)
        assert torch.equal(again["dx"], r["dx"]) and torch.equal(again["dw"], r["dw"])


def test_residual_norm_backward_differences():
    g = gen(11)
    x, w = randn(g, 5, 264).double(), 1 + 0.1 * randn(g, 264).double()
    dy, dvx, dvw = randn(g, 5, 264).double(), randn(g, 5, 264).double(), randn(g, 264).double()
    f = lambda a, b: (norm_ref(a, None, b, torch.float64)[1] * dy).sum()  # noqa: E731
    h = 1e-5
    want_x = (f(x + h * dvx, w) - f(x - h * dvx, w)) / (2 * h)
    want_w = (f(x, w + h * dvw) - f(x, w - h * dvw)) / (2 * h)
    r = gdn.residual_norm_backward(dy.float(), x.float(), w.float(), None, EPS)
    # fp32 inputs and results: 2^-24 a factor, five factors and a 264-term sum
    scale_x = (r["dx"].double().abs() * dvx.abs()).sum()
    scale_w = (r["dw"].double().abs() * dvw.abs()).sum()
    tol = 264 * 2.0 ** -23
    assert abs((r["dx"].double() * dvx).sum() - want_x) <= tol * scale_x + 1e-6 * abs(want_x)
    assert abs((r["dw"].double() * dvw).sum() - want_w) <= tol * scale_w + 1e-6 * abs(want_w)


# ------------------------------------------------------------ quantisation
@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 128), (3, 136), (130, 2048), (257, 1000)])
def test_quantize_fp8(io, rows, cols):
    g = gen(rows + cols)
    x = randn(g, rows, cols, dtype=io)
    x[:, ::17] *= 30
    q, scale = gdn.quantize_fp8(x)
    check_quantised(q, scale, x.double(), 2.0 ** -23)
    qw, sw = gdn.quantize_fp8(x, block_rows=128)
    nr, nc = -(-rows // 128), -(-cols // 128)
    assert sw.shape == (nr, nc)
    for i in range(nr):
        for j in range(nc):
            t = x[128 * i:128 * i + 128, 128 * j:128 * j + 128].double()
            m = t.abs().max()
            within(sw[i, j], m / 448, 2.0 ** -23 * m / 448)
            got = qw[128 * i:128 * i + 128, 128 * j:128 * j + 128].float().double() * sw[i, j].double()
            within(got, t, (2.0 ** -4 + 2.0 ** -22) * t.abs() + 2.0 ** -10 * m / 448 * (1 + 2.0 ** -22))


def e4m3_of(v):
    """e4m3 value nearest to v (64 bits, |v| <= 448), ties to even; and where it is normal."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step, v.abs() >= 2.0 ** -6


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantised_codes_are_the_real_numbers(io, block_rows):
    """Every code is the rounding of 448 x / m itself, values that fp32 leaves
    on or beside the middle between two codes included (among bf16 values the
    exact middle is common).  64 bits hold 448 x exactly and the quotient to
    2^-53, exactly where it is such a middle."""
    g = gen(81)
    x = randn(g, 1024, 1024, dtype=io)
    x[:, ::7] = torch.randint(-56, 57, (1024, x[:, ::7].shape[1]), generator=g, device=DEV).to(io)
    q, scale = gdn.quantize_fp8(x, block_rows=block_rows)
    b = x.double().view(1024 // block_rows, block_rows, 8, 128)
    m = b.abs().amax((1, 3), keepdim=True)
    want, normal = e4m3_of((448 * b / m).view(1024, 1024))
    assert torch.equal(q.double()[normal], want[normal])


@pytest.mark.parametrize("io", [BF16, F32])
def test_norm_codes_are_the_real_numbers(io):
    """The same for the norm, whose root cancels in y / max |y|: s and w with few
    bits put many values on the middle between two codes."""
    g = gen(82)
    x = torch.randint(-120, 121, (2048, 1024), generator=g, device=DEV).to(io) * 2.0 ** -5
    x[::2] = randn(g, 1024, 1024, dtype=io)
    w = torch.randint(1, 29, (1024,), generator=g, device=DEV).float() / 16
    for rows in (2048, 300):
        q, scale, _ = gdn.residual_norm_fp8(x[:rows], w, eps=EPS)
        p = (x[:rows].double() * w.double()).view(rows, 8, 128)
        want, normal = e4m3_of((448 * p / p.abs().amax(-1, keepdim=True)).view(rows, 1024))
        assert torch.equal(q.double()[normal], want[normal])


# ----------------------------------------------------------- 8-bit product
def spread(scale, rows, cols, block_rows):
    s = scale.double()
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols]


def check_linear(tokens, k, n, out_dtype, seed, misaligned=False):
    g = gen(seed)
    x, sx = gdn.quantize_fp8(randn(g, tokens, k, dtype=BF16))
    w, sw = gdn.quantize_fp8(randn(g, n, k, dtype=BF16, scale=k ** -0.5), block_rows=128)
    # scales that differ strongly from block to block, so that a wrong one shows
    sx = sx * torch.exp2(torch.randint(-3, 4, sx.shape, generator=g, device=DEV).float()) * 0.7
    sw = sw * torch.exp2(torch.randint(-3, 4, sw.shape, generator=g, device=DEV).float()) * 1.3
    item = torch.empty(0, dtype=out_dtype).element_size()
    b = Guarded((tokens, n), out_dtype, pad=(256 + 16 // item) if misaligned else 256)
    out = gdn.linear_fp8(x, sx, w, sw, out_dtype, out=b.t)
    xd = x.double() * spread(sx, tokens, k, 1)
    wd = w.double() * spread(sw, n, k, 128)
    ref, S = xd @ wd.T, xd.abs() @ wd.abs().T
    within(out, ref, HALF[out_dtype] * ref.abs() + (2.0 ** -13 + (k / 128 + 3) * 2.0 ** -23) * S,
           (tokens, k, n))
    assert frob(out, ref) <= (2.0 ** -8 if out_dtype == BF16 else 2.0 ** -12)
    b.check()
    assert gdn.device_status() == 0
    return frob(out, ref)


@pytest.mark.parametrize("tokens,k,n", [
    (1, 16, 1), (1, 128, 128), (2, 144, 6), (3, 2048, 12), (17, 256, 4608), (64, 2048, 300),
    (128, 384, 257), (129, 1552, 255), (256, 2048, 512), (300, 640, 1000), (513, 4096, 129),
    (1000, 1040, 2005)])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_linear_fp8(tokens, k, n, out_dtype):
    check_linear(tokens, k, n, out_dtype, tokens + k + n)


@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 31, 33, 64, 65, 100, 127, 128, 255, 257])
@pytest.mark.parametrize("k,n", [(128, 40), (400, 257), (2048, 4608), (5136, 130)])
def test_linear_fp8_few_tokens(tokens, k, n):
    check_linear(tokens, k, n, BF16, tokens * k + n)


def test_linear_fp8_many_tiles_and_unaligned_rows():
    check_linear(4000, 512, 5000, BF16, 5)           # more tiles than CTA pairs
    check_linear(300, 256, 264, BF16, 6, misaligned=True)
    check_linear(300, 256, 264, F32, 6, misaligned=True)


# tiles of 256 and of 128 columns, in one round and in several, rows of the
# result that start on 16 bytes and that do not
@pytest.mark.parametrize("tokens,k,n", [
    (1000, 256, 4608), (1000, 144, 4607), (1500, 400, 2001), (520, 256, 4608), (513, 400, 4095),
    (3001, 144, 2005), (3001, 640, 2008), (9800, 144, 100), (257, 2048, 4500)])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_linear_fp8_tile_widths(tokens, k, n, out_dtype):
    check_linear(tokens, k, n, out_dtype, tokens + 3 * k + n)


def test_linear_fp8_nan_stays_in_its_row():
    g = gen(9)
    x, sx = gdn.quantize_fp8(randn(g, 20, 512, dtype=BF16))
    w, sw = gdn.quantize_fp8(randn(g, 200, 512, dtype=BF16), block_rows=128)
    clean = gdn.linear_fp8(x, sx, w, sw)
    sx[7, 2] = float("nan")
    out = gdn.linear_fp8(x, sx, w, sw)
    assert bool(torch.isnan(out[7]).all())
    keep = [i for i in range(20) if i != 7]
    assert torch.equal(out[keep], clean[keep])


def test_linear_fp8_batch_axes_streams_and_graphs():
    g = gen(10)
    x, sx = gdn.quantize_fp8(randn(g, 2, 3, 256, dtype=BF16))
    w, sw = gdn.quantize_fp8(randn(g, 40, 256, dtype=BF16), block_rows=128)
    out = gdn.linear_fp8(x, sx, w, sw)
    assert out.shape == (2, 3, 40)
    flat = gdn.linear_fp8(x.view(6, 256), sx.view(6, 2), w, sw)
    assert torch.equal(out.view(6, 40), flat)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = torch.empty_like(out)
    gdn.linear_fp8(x, sx, w, sw, out=o2, stream=side)
    side.synchronize()
    assert torch.equal(o2, out)
    graph = torch.cuda.CUDAGraph()
    o3 = torch.zeros_like(out)
    with torch.cuda.graph(graph):
        gdn.linear_fp8(x, sx, w, sw, out=o3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3, out)


# ------------------------------------------------------------ feed-forward
def act_ref(G, act):
    s = torch.sigmoid(G)
    return (G * s, s * (1 + G * (1 - s))) if act == "silu" else (s, s * (1 - s))


def ffn_inputs(tokens, dim, hidden, seed):
    g = gen(seed)
    return (randn(g, tokens, dim, dtype=BF16), randn(g, hidden, dim, dtype=BF16, scale=dim ** -0.5),
            randn(g, hidden, dim, dtype=BF16, scale=dim ** -0.5),
            randn(g, tokens, hidden, dtype=BF16, scale=0.1))


def ffn_terms(x, wg, wu, act):
    """G, U, act, act' and the bounds on the errors of the first three, in 64 bits."""
    xd, gd, ud = x.double(), wg.double(), wu.double()
    c = (x.shape[1] / 16 + 1) * 2.0 ** -23
    G, U = xd @ gd.T, xd @ ud.T
    eG, eU = c * (xd.abs() @ gd.abs().T), c * (xd.abs() @ ud.abs().T)
    a, da = act_ref(G, act)
    ea = 1.1 * eG + 2.0 ** -19 * a.abs() + 2.0 ** -126   # |act'| <= 1.1; its flushed tail
    eda = eG + 2.0 ** -18 * (1 + G.abs()) * torch.sigmoid(G)   # |act''| <= 1/2
    return G, U, a, da, eU, ea, eda


FFN_SHAPES = [(1, 8, 1), (1, 64, 128), (3, 72, 130), (17, 256, 96), (128, 128, 256),
              (130, 520, 300), (257, 1032, 515), (600, 2048, 1000)]


@pytest.mark.parametrize("tokens,dim,hidden", FFN_SHAPES)
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gated_ffn(tokens, dim, hidden, act):
    x, wg, wu, _ = ffn_inputs(tokens, dim, hidden, tokens + dim + hidden)
    b = Guarded((tokens, hidden), BF16)
    h = gdn.gated_ffn(x, wg, wu, act, h=b.t)
    G, U, a, da, eU, ea, _ = ffn_terms(x, wg, wu, act)
    ref = a * U
    within(h, ref, (2.0 ** -8 + 2.0 ** -22) * ref.abs() + 1.01 * (ea * U.abs() + a.abs() * eU), "h")
    b.check()
    assert gdn.device_status() == 0


@pytest.mark.parametrize("tokens", [1, 2, 16, 17, 33, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("dim,hidden", [(64, 64), (200, 65), (2048, 6144), (4104, 131)])
def test_gated_ffn_few_tokens(tokens, dim, hidden):
    x, wg, wu, _ = ffn_inputs(tokens, dim, hidden, tokens * dim + hidden)
    b = Guarded((tokens, hidden), BF16)
    h = gdn.gated_ffn(x, wg, wu, h=b.t)
    G, U, a, _, eU, ea, _ = ffn_terms(x, wg, wu, "silu")
    within(h, a * U, (2.0 ** -8 + 2.0 ** -22) * (a * U).abs()
           + 1.01 * (ea * U.abs() + a.abs() * eU), "h")
    b.check()
    assert gdn.device_status() == 0


def check_ffn_backward(tokens, dim, hidden, act, seed):
    x, wg, wu, dh = ffn_inputs(tokens, dim, hidden, seed)
    r = gdn.gated_ffn_backward(x, wg, wu, dh, act)
    assert gdn.device_status() == 0
    G, U, a, da, eU, ea, eda = ffn_terms(x, wg, wu, act)
    d = dh.double()
    dU, dG = d * a, d * U * da
    edU = 1.01 * d.abs() * ea + 2.0 ** -8 * dU.abs()
    edG = 1.01 * d.abs() * (eU * da.abs() + U.abs() * eda) + (2.0 ** -8 + 2.0 ** -20) * dG.abs()
    xd, gd, ud = x.double(), wg.double(), wu.double()
    dx = dG @ gd + dU @ ud
    cx, cw = (2 * hidden / 16 + 2) * 2.0 ** -23, (tokens / 16 + 1) * 2.0 ** -23
    bx = edG @ gd.abs() + edU @ ud.abs() + cx * (dG.abs() @ gd.abs() + dU.abs() @ ud.abs())
    within(r["dx"], dx, 2.0 ** -8 * dx.abs() + 1.01 * bx + 2.0 ** -133, "dx")
    for name, t, e in (("dw_gate", dG, edG), ("dw_up", dU, edU)):
        ref = t.T @ xd
        b = e.T @ xd.abs() + cw * (t.abs().T @ xd.abs())
        within(r[name], ref, 2.0 ** -8 * ref.abs() + 1.01 * b + 2.0 ** -133, name)
        # roundings of independent signs: the result's and dG's or dU's
        assert frob(r[name], ref) <= 2.0 ** -7, name
    assert frob(r["dx"], dx) <= 2.0 ** -7
    return x, wg, wu, dh, r


@pytest.mark.parametrize("tokens,dim,hidden", FFN_SHAPES + [
    (1, 2048, 40), (700, 264, 2731),
    # few tiles with a long inner axis: dx, the weight gradients, both in parts
    (250, 520, 6000), (5000, 264, 300), (1111, 1032, 2731), (3000, 72, 2100)])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gated_ffn_backward(tokens, dim, hidden, act):
    x, wg, wu, dh, r = check_ffn_backward(tokens, dim, hidden, act, 7 * tokens + dim + hidden)
    ws = torch.empty(gdn.gated_ffn_backward_workspace_size(tokens, dim, hidden),
                     dtype=torch.uint8, device=DEV).fill_(0xFF)   # NaN wherever it is read unwritten
    again = gdn.gated_ffn_backward(x, wg, wu, dh, act, workspace=ws)
    for k in r:
        assert torch.equal(r[k], again[k]), k


def test_gated_ffn_many_tiles():
    x, wg, wu, _ = ffn_inputs(3000, 256, 5000, 21)      # more tiles than CTA pairs
    h = gdn.gated_ffn(x, wg, wu)
    G, U, a, _, eU, ea, _ = ffn_terms(x, wg, wu, "silu")
    within(h, a * U, 2.0 ** -7.99 * (a * U).abs() + 1.01 * (ea * U.abs() + a.abs() * eU))
    check_ffn_backward(2500, 1000, 3000, "silu", 22)
    assert gdn.device_status() == 0


# tiles of 256 columns where they fill the last round, of 192 elsewhere; rows of
# the result that start on 16 bytes and that do not
@pytest.mark.parametrize("tokens,dim,hidden", [
    (777, 64, 8000), (777, 64, 8001), (300, 72, 6000), (300, 72, 6001), (513, 136, 2053),
    (255, 64, 9700), (255, 64, 9699), (1000, 72, 97), (1000, 72, 33), (1000, 72, 95)])
def test_gated_ffn_tile_widths(tokens, dim, hidden):
    x, wg, wu, _ = ffn_inputs(tokens, dim, hidden, 3 * tokens + hidden)
    b = Guarded((tokens, hidden), BF16)
    h = gdn.gated_ffn(x, wg, wu, h=b.t)
    G, U, a, _, eU, ea, _ = ffn_terms(x, wg, wu, "silu")
    within(h, a * U, (2.0 ** -8 + 2.0 ** -22) * (a * U).abs()
           + 1.01 * (ea * U.abs() + a.abs() * eU), "h")
    b.check()
    check_ffn_backward(tokens, dim, hidden, "silu", 5 * tokens + hidden)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gated_ffn_backward_differences(act):
    x, wg, wu, dh = ffn_inputs(33, 64, 48, 31)
    r = gdn.gated_ffn_backward(x, wg, wu, dh, act)
    v = [randn(gen(32 + i), *t.shape).double() for i, t in enumerate((x, wg, wu))]
    base = [t.double() for t in (x, wg, wu)]

    def loss(i, h):
        t = [b + (h * v[j] if j == i else 0) for j, b in enumerate(base)]
        return (act_ref(t[0] @ t[1].T, act)[0] * (t[0] @ t[2].T) * dh.double()).sum()

    for i, name in enumerate(("dx", "dw_gate", "dw_up")):
        want = (loss(i, 1e-5) - loss(i, -1e-5)) / 2e-5
        got = (r[name].double() * v[i]).sum()
        # two bf16 roundings of independent signs in every term
        tol = 4 * 2.0 ** -8 * (r[name].double() * v[i]).norm()
        assert abs(got - want) <= tol, (name, float(got), float(want))


def test_gated_ffn_infinite_and_empty_inputs():
    x, wg, wu, dh = ffn_inputs(5, 64, 40, 41)
    clean = gdn.gated_ffn(x, wg, wu)
    x[2, 3] = float("inf")
    h = gdn.gated_ffn(x, wg, wu)
    keep = [0, 1, 3, 4]
    assert torch.equal(h[keep], clean[keep]) and not bool(torch.isfinite(h[2]).all())
    e = x[:0]
    assert gdn.gated_ffn(e, wg, wu).shape == (0, 40)
    r = gdn.gated_ffn_backward(e, wg, wu, dh[:0])
    assert r["dx"].shape == (0, 64) and float(r["dw_gate"].abs().max()) == 0
    assert float(r["dw_up"].abs().max()) == 0
    # far in the tails of the gate
    big = torch.full((2, 64), 300.0, dtype=BF16, device=DEV)
    one = torch.ones(8, 64, dtype=BF16, device=DEV)
    assert bool(torch.isfinite(gdn.gated_ffn(big, one, one)).all())
    assert float(gdn.gated_ffn(-big, one, one).abs().max()) == 0


# ------------------------------------------------- graphs, streams, workspaces
def training_step(t, ws=None):
    """Norm, feed-forward and both gradients on fixed tensors."""
    y, s = gdn.residual_norm(t["x"], t["w"], t["r"], EPS)
    h = gdn.gated_ffn(y, t["wg"], t["wu"])
    f = gdn.gated_ffn_backward(y, t["wg"], t["wu"], t["dh"],
                               workspace=None if ws is None else ws[0])
    n = gdn.residual_norm_backward(f["dx"], s, t["w"], t["r"], EPS,
                                   workspace=None if ws is None else ws[1])
    return [y, s, h, *f.values(), *n.values()]


def step_tensors(seed, tokens=300, dim=264, hidden=700):
    g = gen(seed)
    x, wg, wu, dh = ffn_inputs(tokens, dim, hidden, seed)
    return dict(x=x, r=randn(g, tokens, dim, dtype=BF16), w=1 + 0.1 * randn(g, dim), wg=wg, wu=wu,
                dh=dh)


@pytest.mark.parametrize("own_workspace", [False, True])
def test_training_step_in_a_graph(own_workspace):
    t, other = step_tensors(51), step_tensors(52)
    want = [training_step(t), training_step(other)]
    tokens, dim, hidden = 300, 264, 700
    sizes = (gdn.gated_ffn_backward_workspace_size(tokens, dim, hidden),
             gdn.residual_norm_backward_workspace_size(tokens, dim))
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes] if own_workspace else None
    live = {k: v.clone() for k, v in t.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = training_step(live, ws)
    for source, ref in ((t, want[0]), (other, want[1]), (t, want[0])):
        for k, v in source.items():
            live[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
    assert gdn.device_status() == 0


def test_streams_side_by_side():
    """The same calls on two streams at once give each stream's own results."""
    sets = [step_tensors(61), step_tensors(62, tokens=1500, dim=512, hidden=900)]
    g = gen(63)
    q = [gdn.quantize_fp8(randn(g, n, 512, dtype=BF16)) for n in (40, 700)]
    w = gdn.quantize_fp8(randn(g, 300, 512, dtype=BF16), block_rows=128)
    want = [training_step(t) + [gdn.linear_fp8(*a, *w)] for t, a in zip(sets, q)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(training_step(sets[i]) + [gdn.linear_fp8(*q[i], *w)])
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)
    assert gdn.device_status() == 0


def test_workspace_stays_inside():
    tokens, dim, hidden = 1111, 264, 2731          # weight gradients and dx in parts
    x, wg, wu, dh = ffn_inputs(tokens, dim, hidden, 71)
    n = gdn.gated_ffn_backward_workspace_size(tokens, dim, hidden)
    b = Guarded((n,), torch.uint8)
    gdn.gated_ffn_backward(x, wg, wu, dh, workspace=b.t)
    b.check()
    n = gdn.residual_norm_backward_workspace_size(tokens, dim)
    b = Guarded((n,), torch.uint8)
    gdn.residual_norm_backward(x, x, torch.ones(dim, device=DEV), workspace=b.t)
    b.check()
    with pytest.raises(gdn.GDNError):
        gdn.residual_norm_backward(x, x, torch.ones(dim, device=DEV), workspace=b.t[:-256])
