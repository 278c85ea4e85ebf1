"""Attention over prompts against the formula in 64 bits.

Tolerance, element by element, with A = sum_j p_j |v_j| (p normalised): the result's rounding
2^-8 |o| and each probability's rounding to bf16, 2^-8 A; the exponents' errors, those of a sum of
d <= 128 fp32 products and of 2^x, are under 2^-16 (1 + size) of A with size = scale max |q| |k|
(128 products of 2^-24 relative error each, of a sum of magnitudes at most size, make 2^-17 size).
lse: the same exponents' error, absolute."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
BAD_SEQLENS = 6


def cu(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def inputs(tq, tk, H, kv, d, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return ((scale * new(tq, H, d)).to(BF16), new(tk, kv, d).to(BF16), new(tk, kv, d).to(BF16))


def formula(q, k, v, scale):
    """One sequence in 64 bits: out, lse, A, size [heads, ..]."""
    lq, H, d = q.shape
    lk, kv = k.shape[:2]
    q, k, v = (t.double().transpose(0, 1) for t in (q, k, v))
    k, v = (t.repeat_interleave(H // kv, 0) for t in (k, v))
    s = scale * q @ k.transpose(1, 2)
    see = torch.arange(lk, device="cuda") <= torch.arange(lq, device="cuda")[:, None] + lk - lq
    s = s.masked_fill(~see, float("-inf"))
    lse = s.logsumexp(-1)
    p = torch.exp(s - lse.masked_fill(lse.isneginf(), 0)[..., None])
    kmax = k.norm(dim=-1).amax(-1)[:, None] if lk else torch.zeros(H, 1, device="cuda").double()
    size = scale * q.norm(dim=-1) * kmax
    return p @ v, lse, p @ v.abs(), size


def verify(q, k, v, out, lse, ql, kl, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    a = b = 0
    for lq, lk in zip(ql, kl):
        o, want, A, size = formula(q[a:a + lq], k[b:b + lk], v[b:b + lk], scale)
        got = out[a:a + lq].double().transpose(0, 1)
        tol = 2.0 ** -8 * 1.01 * (o.abs() + A) + A * (2.0 ** -16 * (1 + size))[..., None]
        assert ((got - o).abs() <= tol).all(), (lq, lk, float(((got - o).abs() - tol).max()))
        gl = lse[a:a + lq].double().t()
        none = want.isneginf()
        assert torch.equal(gl.isneginf(), none) and (got[none] == 0).all()
        off = (gl - want)[~none].abs()
        assert (off <= (2.0 ** -16 * (1 + size))[~none]).all(), float(off.max())
        a, b = a + lq, b + lk


RAGGED = [1, 127, 128, 129, 0, 64, 33, 300, 255, 257, 2]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 4), (1, 3), (3, 7), (1, 16), (2, 5), (1, 128),
                                      (1, 65)])
def test_packed_lengths_and_groups(gdn_lib, d, kv, group):
    gdn = gdn_lib
    H, n = kv * group, sum(RAGGED)
    q, k, v = inputs(n, n, H, kv, d, group)
    out, lse = gdn.attention_prefill(q, k, v, cu(RAGGED))
    verify(q, k, v, out, lse, RAGGED, RAGGED)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("d,kv,group", [(64, 2, 3), (128, 2, 4), (128, 1, 1)])
@pytest.mark.parametrize("ql,kl", [
    ([17], [1200]), ([1], [1]), ([1], [129]), ([1, 1, 1], [127, 128, 4000]),
    ([300, 5, 0, 40], [100, 0, 7, 40]),            # rows that see nothing
    ([200, 129], [1, 128]), ([64, 500], [64 + 128, 500 + 77]), ([1000], [1000]), ([5, 6], [0, 0])])
def test_context_and_empty_rows(gdn_lib, ql, kl, d, kv, group):
    gdn = gdn_lib
    q, k, v = inputs(sum(ql), sum(kl), kv * group, kv, d, sum(kl))
    out, lse = gdn.attention_prefill(q, k, v, cu(ql), cu(kl))
    verify(q, k, v, out, lse, ql, kl)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("B,tq,tk,d", [(3, 200, 200, 64), (2, 77, 333, 128), (5, 1, 1, 128),
                                       (2, 50, 20, 64), (1, 2500, 2500, 128)])
def test_dense_batches(gdn_lib, B, tq, tk, d):
    gdn = gdn_lib
    q, k, v = inputs(B * tq, B * tk, 6, 2, d)
    out, lse = gdn.attention_prefill(q.view(B, tq, 6, d), k.view(B, tk, 2, d), v.view(B, tk, 2, d))
    assert out.shape == (B, tq, 6, d) and lse.shape == (B, tq, 6)
    verify(q, k, v, out.flatten(0, 1), lse.flatten(0, 1), [tq] * B, [tk] * B)
    # (packed, a sequence's keys may be cut into other parts)
    verify(q, k, v, *gdn.attention_prefill(q, k, v, cu([tq] * B), cu([tk] * B)), [tq] * B, [tk] * B)


@pytest.mark.parametrize("d", [64, 128])
def test_growing_maxima_and_scales(gdn_lib, d):
    """Scores that grow along the keys, so that sums are rescaled again and again; sharp and flat
    ones; another scale."""
    gdn = gdn_lib
    n = 1500
    q, k, v = inputs(n, n, 4, 2, d)
    k = (k * torch.linspace(0.05, 30, n, device="cuda")[:, None, None]).to(BF16)
    for scale in (None, 0.5, 1e-3):
        out, lse = gdn.attention_prefill(q, k, v, cu([n]), scale=scale)
        verify(q, k, v, out, lse, [n], [n], scale)
    zero = torch.zeros_like(q)
    out, lse = gdn.attention_prefill(zero, k, v, cu([n]))
    verify(zero, k, v, out, lse, [n], [n])
    falling = k.flip(0).contiguous()
    out, lse = gdn.attention_prefill(q, falling, v, cu([n]))
    verify(q, falling, v, out, lse, [n], [n])


def test_slices_of_a_packed_projection(gdn_lib):
    gdn = gdn_lib
    n, H, kv, d = 333, 6, 2, 64
    x = torch.randn(n, (H + 2 * kv) * d + 8, device="cuda").to(BF16)
    q = x[:, 8:8 + H * d].unflatten(1, (H, d))
    k = x[:, 8 + H * d:8 + (H + kv) * d].unflatten(1, (kv, d))
    v = x[:, 8 + (H + kv) * d:].unflatten(1, (kv, d))
    lens = [200, 133]
    out, lse = gdn.attention_prefill(q, k, v, cu(lens))
    verify(q, k, v, out, lse, lens, lens)
    same = gdn.attention_prefill(q.contiguous(), k.contiguous(), v.contiguous(), cu(lens))
    assert torch.equal(out, same[0]) and torch.equal(lse, same[1])


@pytest.mark.parametrize("d", [64, 128])
def test_other_sequences_stay_out(gdn_lib, d):
    """NaN and infinities in one sequence change no bit of another's results; nothing behind the
    results is written."""
    gdn = gdn_lib
    lens = [100, 130, 60, 257]
    n = sum(lens)
    q, k, v = inputs(n, n, 4, 2, d)
    c = cu(lens)
    out, lse = gdn.attention_prefill(q, k, v, c)
    for t, bad in ((q, float("inf")), (k, float("nan")), (v, float("inf"))):
        x = t.clone()
        x[100:230] = bad
        args = [x if y is t else y for y in (q, k, v)]
        room, lroom = torch.full((n + 9, 4, d), 7.0, device="cuda", dtype=BF16), \
            torch.full((n + 9, 4), 7.0, device="cuda")
        o, s = gdn.attention_prefill(*args, c, out=room[:n], lse=lroom[:n])
        for part in (slice(0, 100), slice(230, n)):
            assert torch.equal(o[part], out[part]) and torch.equal(s[part], lse[part])
        assert (room[n:] == 7).all() and (lroom[n:] == 7).all()
        assert o[100:230].isnan().any()
    # a value of the own sequence reaches the rows of its tile of keys, no earlier ones
    x = v.clone()
    x[230 + 60 + 200] = float("nan")
    o, _ = gdn.attention_prefill(q, k, x, c)
    assert torch.equal(o[:290 + 128], out[:290 + 128]) and o[290 + 200:].isnan().any()


def test_many_sequences(gdn_lib):
    gdn, rng = gdn_lib, random.Random(3)
    ql = [rng.choice([0, 1, 3, 40, 130]) for _ in range(1500)]
    kl = [max(0, n + rng.choice([0, 0, 5, -2, 128])) for n in ql]
    q, k, v = inputs(sum(ql), sum(kl), 3, 1, 64)
    out, lse = gdn.attention_prefill(q, k, v, cu(ql), cu(kl))
    at = [sum(ql[:i]) for i in range(len(ql))]
    ak = [sum(kl[:i]) for i in range(len(kl))]
    for i in list(range(0, 1500, 40)) + [1499]:
        a, b = at[i], ak[i]
        verify(q[a:a + ql[i]], k[b:b + kl[i]], v[b:b + kl[i]], out[a:a + ql[i]], lse[a:a + ql[i]],
               [ql[i]], [kl[i]])
    assert gdn.device_status() == 0


@pytest.mark.parametrize("bad", [[0, 200, 100, 300], [1, 100, 200, 300], [0, 100, 200, 299],
                                 [0, -100, 200, 300]])
@pytest.mark.parametrize("which", ["q", "k"])
def test_malformed_sequences_write_nothing(gdn_lib, bad, which):
    gdn = gdn_lib
    q, k, v = inputs(300, 300, 2, 1, 64)
    good, wrong = cu([100, 100, 100]), torch.tensor(bad, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7), torch.full((300, 2), 7.0, device="cuda")
    args = (wrong, good) if which == "q" else (good, wrong)
    gdn.attention_prefill(q, k, v, *args, out=out, lse=lse)
    assert gdn.device_status() == BAD_SEQLENS
    assert (out == 7).all() and (lse == 7).all()


def test_streams_and_graphs(gdn_lib):
    """Two captured calls side by side, and the same bits every time."""
    gdn = gdn_lib
    n = 700
    jobs = []
    for i in range(2):
        q, k, v = inputs(n, n, 4, 2, 128, i)
        c, st = cu([n - 300 - i, 300 + i]), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            want = gdn.attention_prefill(q, k, v, c)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                got = gdn.attention_prefill(q, k, v, c)
        jobs.append((st, graph, want, got, (q, k, v, c)))
    for _ in range(10):
        for st, graph, _, got, _ in jobs:
            with torch.cuda.stream(st):
                got[0].zero_()
                graph.replay()
    torch.cuda.synchronize()
    for _, _, want, got, _ in jobs:
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_nothing_to_do(gdn_lib):
    gdn = gdn_lib
    q, k, v = inputs(0, 5, 4, 2, 64)
    out, lse = gdn.attention_prefill(q, k, v, cu([0]), cu([5]))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    q, k, v = inputs(5, 0, 4, 2, 64)
    out, lse = gdn.attention_prefill(q, k, v, cu([5]), cu([0]))
    assert (out == 0).all() and lse.isneginf().all()
    assert gdn.device_status() == 0


@pytest.mark.parametrize("n", [300, 3000])
def test_scores_of_minus_infinity(gdn_lib, n):
    """Keys whose scores are -inf count for nothing, however many come before the first finite one."""
    d, m = 128, n - 20
    q = torch.ones(n, 2, d, device="cuda", dtype=BF16)
    k = torch.full((n, 1, d), -10.0, device="cuda", dtype=BF16)
    k[:m] = -float("inf")
    g = torch.Generator(device="cuda").manual_seed(8)
    v = torch.randn(n, 1, d, generator=g, device="cuda").to(BF16)
    out, lse = gdn_lib.attention_prefill(q, k, v)
    assert lse[:m].isneginf().all() and (out[:m] == 0).all()
    o, want = gdn_lib.attention_prefill(q[m:], k[m:], v[m:])
    # (all finite scores are equal: the probabilities are 1, the sums' order apart)
    assert (out[m:].float() - o.float()).abs().max() <= 2.0 ** -7 * v.abs().max()
    assert (lse[m:] - want).abs().max() <= 2.0 ** -16 * (1 + want.abs().max())
    assert gdn_lib.device_status() == 0


def test_more_tiles_than_levels(gdn_lib):
    """128 heads on one: tiles of two queries, more of them than the list tells apart."""
    g = torch.Generator(device="cuda").manual_seed(21)
    n, d = 5000, 64
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(BF16) for h in (128, 1, 1))
    out, lse = gdn_lib.attention_prefill(q, k, v)
    for a, b in ((0, 200), (2500, 2540), (n - 40, n)):
        verify(q[a:b], k[:b], v[:b], out[a:b], lse[a:b], [b - a], [b])
    assert gdn_lib.device_status() == 0


def test_tensors_of_more_than_2_31_elements(gdn_lib):
    g = torch.Generator(device="cuda").manual_seed(22)
    H, d, lens = 64, 128, [64] * 4200 + [200]
    T = sum(lens)
    q, k, v = (torch.randn(T, H, d, generator=g, device="cuda", dtype=BF16) for _ in range(3))
    c = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    out, lse = gdn_lib.attention_prefill(q, k, v, c)
    assert q.numel() > 2 ** 31
    for a, b in ((0, 64), (64 * 4100, 64 * 4101), (T - 200, T)):
        verify(q[a:b], k[a:b], v[a:b], out[a:b], lse[a:b], [b - a], [b - a])
    assert gdn_lib.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ql,kl", [([20], [9000]), ([1], [1000]), ([64, 3], [700, 40]), ([130], [130]),
                                   ([200, 0, 90], [3000, 5, 2000]), ([1000], [1000])])
def test_keys_in_parts(gdn_lib, ql, kl, d):
    """Few tiles behind many keys: the parts of a tile's keys are joined; the same bits every time."""
    q, k, v = inputs(sum(ql), sum(kl), 6, 2, d, seed=sum(kl))
    out, lse = gdn_lib.attention_prefill(q, k, v, cu(ql), cu(kl))
    verify(q, k, v, out, lse, ql, kl)
    for _ in range(3):
        again = gdn_lib.attention_prefill(q, k, v, cu(ql), cu(kl))
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert gdn_lib.device_status() == 0
