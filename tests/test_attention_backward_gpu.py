"""Gradients of the attention over prompts against the formula in 64 bits and against differences.

Tolerance, element by element: with e = 2^-16 (1 + size), size = scale max |q| |k| (the exponents'
error, see the forward tests), P carries e P, and its rounding to bf16 2^-8 P; dS = P (dP - D)
carries its rounding and e, (2^-8 + e) |dS|, and the fp32 sums of dP and D, 2^-16 P |do| (|v| + |o|).
A gradient then carries the sum of these over its products, a sum's own error (2^-12 of the sum
of magnitudes, for n <= 4096 terms of 2^-24 each) and its rounding 2^-8.

One absolute term: 2^x gives 0 where P < 2^-126 (fp32's smallest normal number; the tests' scores
lie hundreds of powers of two apart), and bf16 holds nothing below 2^-133.  A term that is lost so
is under 2^-126 times |do| (|v| + |o|) |k| scale < 2^14 here, and a sum has at most 2^12 of them:
TINY = 2^-100."""
import random

import pytest
import torch

from test_attention_prefill_gpu import cu, inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
BAD_SEQLENS = 6
TINY = 2.0 ** -100


def formula(q, k, v, out, lse, dout, scale):
    """One sequence: (gradient, tolerance) of q, k, v."""
    lq, H, d = q.shape
    lk, kv = k.shape[:2]
    G = H // kv
    q, k, v, out, do = (t.double().transpose(0, 1) for t in (q, k, v, out, dout))
    kk, vv = (t.repeat_interleave(G, 0) for t in (k, v))
    lse = lse.double().t()
    s = scale * q @ kk.transpose(1, 2)
    see = torch.arange(lk, device="cuda") <= torch.arange(lq, device="cuda")[:, None] + lk - lq
    P = torch.exp(s - lse.masked_fill(lse.isneginf(), 0)[..., None]).masked_fill(~see, 0)
    dS = P * (do @ vv.transpose(1, 2) - (do * out).sum(-1, keepdim=True))
    kmax, vmax = (t.norm(dim=-1).amax(-1)[:, None] if lk else torch.zeros(H, 1, device="cuda").double()
                  for t in (kk, vv))
    e = (2.0 ** -16 * (1 + scale * q.norm(dim=-1) * kmax))[..., None]
    dn = do.norm(dim=-1)
    dS_off = (2.0 ** -8 * 1.01 + e + 2.0 ** -12) * dS.abs() + \
        2.0 ** -16 * P * (dn * (vmax + out.norm(dim=-1)))[..., None]
    P_off = (2.0 ** -8 * 1.01 + e + 2.0 ** -12) * P
    fold = lambda t: t.view(kv, G, lk, d).sum(1)  # noqa: E731
    dq, dq_off = scale * dS @ kk, scale * dS_off @ kk.abs()
    dk, dk_off = (fold(scale * x.transpose(1, 2) @ y) for x, y in ((dS, q), (dS_off, q.abs())))
    dv, dv_off = (fold(x.transpose(1, 2) @ y) for x, y in ((P, do), (P_off, do.abs())))
    return [(g.transpose(0, 1), (off + 2.0 ** -8 * g.abs() + TINY).transpose(0, 1))
            for g, off in ((dq, dq_off), (dk, dk_off), (dv, dv_off))]


def verify(q, k, v, out, lse, dout, got, ql, kl, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    a = b = 0
    for lq, lk in zip(ql, kl):
        x, y = slice(a, a + lq), slice(b, b + lk)
        want = formula(q[x], k[y], v[y], out[x], lse[x], dout[x], scale)
        for (g, tol), name, part in zip(want, ("dq", "dk", "dv"), (x, y, y)):
            off = (got[name][part].double() - g).abs()
            assert (off <= tol).all(), (name, lq, lk, float((off - tol).max()))
        a, b = a + lq, b + lk


def step(gdn, q, k, v, c, ck=None, scale=None, seed=9):
    out, lse = gdn.attention_prefill(q, k, v, c, ck, scale)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dout = torch.randn(q.shape, generator=g, device="cuda").to(BF16)
    return out, lse, dout, gdn.attention_prefill_backward(q, k, v, out, lse, dout, c, ck, scale)


RAGGED = [1, 127, 128, 129, 0, 64, 33, 300, 255, 257, 2]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 4), (1, 3), (3, 7), (1, 16), (2, 5), (1, 128),
                                      (1, 65)])
def test_packed_lengths_and_groups(gdn_lib, d, kv, group):
    gdn = gdn_lib
    q, k, v = inputs(sum(RAGGED), sum(RAGGED), kv * group, kv, d, group)
    c = cu(RAGGED)
    out, lse, dout, got = step(gdn, q, k, v, c)
    verify(q, k, v, out, lse, dout, got, RAGGED, RAGGED)
    ws = torch.full((gdn.attention_prefill_backward_workspace_size(len(RAGGED), len(q), kv * group, kv,
                                                                   d, varlen=True),), 255,
                    dtype=torch.uint8, device="cuda")
    again = gdn.attention_prefill_backward(q, k, v, out, lse, dout, c, workspace=ws)
    assert all(torch.equal(got[n], again[n]) for n in got)      # the same bits every time
    assert gdn.device_status() == 0


@pytest.mark.parametrize("d,kv,group", [(64, 2, 3), (128, 2, 4), (128, 1, 1)])
@pytest.mark.parametrize("ql,kl", [
    ([17], [1200]), ([1], [1]), ([1], [129]), ([1, 1, 1], [127, 128, 4000]),
    ([300, 5, 0, 40], [100, 0, 7, 40]),            # rows that see nothing, keys that none sees
    ([200, 129], [1, 128]), ([64, 500], [64 + 128, 500 + 77]), ([1000], [1000]), ([5, 6], [0, 0]),
    ([0, 0], [5, 140])])
def test_context_and_empty_rows(gdn_lib, ql, kl, d, kv, group):
    gdn = gdn_lib
    q, k, v = inputs(sum(ql), sum(kl), kv * group, kv, d, sum(kl))
    out, lse, dout, got = step(gdn, q, k, v, cu(ql), cu(kl))
    verify(q, k, v, out, lse, dout, got, ql, kl)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("B,tq,tk,d", [(3, 200, 200, 64), (2, 77, 333, 128), (5, 1, 1, 128),
                                       (2, 50, 20, 64), (1, 2500, 2500, 128)])
def test_dense_batches(gdn_lib, B, tq, tk, d):
    gdn = gdn_lib
    q, k, v = inputs(B * tq, B * tk, 6, 2, d)
    shaped = q.view(B, tq, 6, d), k.view(B, tk, 2, d), v.view(B, tk, 2, d)
    out, lse, dout, got = step(gdn, *shaped, None)
    flat = {n: t.flatten(0, 1) for n, t in got.items()}
    out, lse, dout = (t.flatten(0, 1) for t in (out, lse, dout))
    verify(q, k, v, out, lse, dout, flat, [tq] * B, [tk] * B)
    packed = gdn.attention_prefill_backward(q, k, v, out, lse, dout, cu([tq] * B), cu([tk] * B))
    # (packed, a key's queries may be cut into other parts)
    verify(q, k, v, out, lse, dout, packed, [tq] * B, [tk] * B)


@pytest.mark.parametrize("d", [64, 128])
def test_sharp_scores_and_scales(gdn_lib, d):
    gdn = gdn_lib
    n = 700
    q, k, v = inputs(n, n, 4, 2, d)
    k = (k * torch.linspace(0.05, 10, n, device="cuda")[:, None, None]).to(BF16)
    for scale in (None, 0.4, 1e-3):
        out, lse, dout, got = step(gdn, q, k, v, cu([n]), scale=scale)
        verify(q, k, v, out, lse, dout, got, [n], [n], scale)


def test_slices_of_a_packed_projection(gdn_lib):
    gdn = gdn_lib
    n, H, kv, d = 333, 6, 2, 64
    x = torch.randn(n, (H + 2 * kv) * d + 8, device="cuda").to(BF16)
    q = x[:, 8:8 + H * d].unflatten(1, (H, d))
    k = x[:, 8 + H * d:8 + (H + kv) * d].unflatten(1, (kv, d))
    v = x[:, 8 + (H + kv) * d:].unflatten(1, (kv, d))
    c = cu([200, 133])
    out, lse, dout, got = step(gdn, q, k, v, c)
    verify(q, k, v, out, lse, dout, got, [200, 133], [200, 133])
    assert got["dq"].is_contiguous() and got["dk"].is_contiguous()


@pytest.mark.parametrize("d", [64, 128])
def test_other_sequences_stay_out(gdn_lib, d):
    """NaN and infinities of one sequence, in any tensor, change no bit of another's gradients;
    nothing behind the results is written."""
    gdn = gdn_lib
    lens = [100, 130, 60, 257]
    n = sum(lens)
    q, k, v = inputs(n, n, 3, 1, d)
    c = cu(lens)
    out, lse, dout, got = step(gdn, q, k, v, c)
    names = dict(q=q, k=k, v=v, out=out, lse=lse, dout=dout)
    for name, bad in (("q", float("inf")), ("k", float("nan")), ("v", float("inf")),
                      ("out", float("nan")), ("lse", float("nan")), ("dout", float("inf"))):
        args = dict(names, **{name: names[name].clone()})
        args[name][100:230] = bad
        other = gdn.attention_prefill_backward(**args, cu_seqlens=c)
        for g in got:
            for part in (slice(0, 100), slice(230, n)):
                assert torch.equal(other[g][part], got[g][part]), (name, g)


def test_against_differences(gdn_lib):
    """The formula itself: the change of <dout, out> along random directions (64 bits)."""
    torch.manual_seed(0)
    from test_attention_prefill_gpu import formula as forward
    lq, lk, H, kv, d = 20, 33, 4, 2, 64
    q, k, v = (torch.randn(n, h, d, device="cuda").double() for n, h in ((lq, H), (lk, kv), (lk, kv)))
    scale, dout = d ** -0.5, torch.randn(lq, H, d, device="cuda").double()
    loss = lambda *t: (forward(*t, scale)[0].transpose(0, 1) * dout).sum()  # noqa: E731
    o, lse, _, _ = forward(q, k, v, scale)
    want = formula(q, k, v, o.transpose(0, 1), lse.t(), dout, scale)
    for i in range(3):
        x = [q, k, v]
        u = torch.randn_like(x[i])
        h = 1e-5
        up, down = ([t + s * h * u if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        slope = (loss(*up) - loss(*down)) / (2 * h)
        assert abs(float(slope - (want[i][0] * u).sum())) <= 1e-6 * float(u.abs().sum())


def test_many_sequences(gdn_lib):
    gdn, rng = gdn_lib, random.Random(3)
    ql = [rng.choice([0, 1, 3, 40, 130]) for _ in range(1500)]
    kl = [max(0, n + rng.choice([0, 0, 5, -2, 128])) for n in ql]
    q, k, v = inputs(sum(ql), sum(kl), 3, 1, 64)
    out, lse, dout, got = step(gdn, q, k, v, cu(ql), cu(kl))
    for i in list(range(0, 1500, 40)) + [1499]:
        x = slice(sum(ql[:i]), sum(ql[:i + 1]))
        y = slice(sum(kl[:i]), sum(kl[:i + 1]))
        part = dict(dq=got["dq"][x], dk=got["dk"][y], dv=got["dv"][y])
        verify(q[x], k[y], v[y], out[x], lse[x], dout[x], part, [ql[i]], [kl[i]])
    assert gdn.device_status() == 0


@pytest.mark.parametrize("bad", [[0, 200, 100, 300], [1, 100, 200, 300], [0, 100, 200, 299]])
def test_malformed_sequences_are_flagged(gdn_lib, bad):
    gdn = gdn_lib
    q, k, v = inputs(300, 300, 2, 1, 64)
    out, lse, dout, got = step(gdn, q, k, v, cu([100, 100, 100]))
    wrong = torch.tensor(bad, dtype=torch.int32, device="cuda")
    gdn.attention_prefill_backward(q, k, v, out, lse, dout, wrong)
    assert gdn.device_status() == BAD_SEQLENS


def test_a_training_step_in_a_graph(gdn_lib):
    """Forward and backward captured on two streams and replayed side by side, the inputs changed
    in between."""
    gdn = gdn_lib
    n, jobs = 500, []
    for i in range(2):
        q, k, v = inputs(n, n, 4, 2, 128, i)
        c, st = cu([n - 300 - i, 300 + i]), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            step(gdn, q, k, v, c)
            dout = torch.randn_like(q)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                out, lse = gdn.attention_prefill(q, k, v, c)
                got = gdn.attention_prefill_backward(q, k, v, out, lse, dout, c)
        jobs.append((st, graph, q, k, v, c, dout, out, lse, got))
    for _ in range(5):
        for st, graph, q, *_ in jobs:
            with torch.cuda.stream(st):
                q.mul_(1.25)
                graph.replay()
    torch.cuda.synchronize()
    for _, _, q, k, v, c, dout, out, lse, got in jobs:
        o, s = gdn.attention_prefill(q, k, v, c)
        want = gdn.attention_prefill_backward(q, k, v, o, s, dout, c)
        assert torch.equal(o, out) and torch.equal(s, lse)
        assert all(torch.equal(want[x], got[x]) for x in want)
    assert gdn.device_status() == 0


def test_more_tiles_than_levels(gdn_lib):
    """128 heads on one: tiles of a query, more of them than the list tells apart."""
    g = torch.Generator(device="cuda").manual_seed(21)
    n, d, H = 5000, 64, 128
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(BF16) for h in (H, 1, 1))
    out, lse, dout, got = step(gdn_lib, q, k, v, None)
    dk, dk_off, dv, dv_off = (torch.zeros(n, 1, d, device="cuda").double() for _ in range(4))
    for h in range(H):
        x = slice(h, h + 1)
        (dq, tol), *kv = formula(q[:, x], k, v, out[:, x], lse[:, x], dout[:, x], d ** -0.5)
        assert ((got["dq"][:, x].double() - dq).abs() <= tol).all(), h
        for total, part in zip((dk, dk_off, dv, dv_off), (t for pair in kv for t in pair)):
            total += part
    assert ((got["dk"].double() - dk).abs() <= dk_off).all()
    assert ((got["dv"].double() - dv).abs() <= dv_off).all()
    assert gdn_lib.device_status() == 0


def test_tensors_of_more_than_2_31_elements(gdn_lib):
    g = torch.Generator(device="cuda").manual_seed(22)
    H, d, lens = 64, 128, [64] * 4200 + [200]
    T = sum(lens)
    q, k, v, dout = (torch.randn(T, H, d, generator=g, device="cuda", dtype=BF16) for _ in range(4))
    c = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    out, lse = gdn_lib.attention_prefill(q, k, v, c)
    got = gdn_lib.attention_prefill_backward(q, k, v, out, lse, dout, c)
    for a, b in ((0, 64), (64 * 4100, 64 * 4101), (T - 200, T)):
        verify(q[a:b], k[a:b], v[a:b], out[a:b], lse[a:b], dout[a:b], {n: t[a:b] for n, t in got.items()},
               [b - a], [b - a])
    assert gdn_lib.device_status() == 0


def test_few_rows_keep_the_results_rounding(gdn_lib):
    """With few rows P and dS have two bf16 terms: 2^-16 of each is lost, and of the gradients only
    what their own rounding loses (with one term 1.4 times as much).  In norm, an eighth of that is
    room for the values that the rounding meets being others than the formula's."""
    g = torch.Generator(device="cuda").manual_seed(31)
    for n, H, kv, d in ((40, 4, 2, 64), (130, 6, 3, 128), (300, 8, 8, 64)):
        q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(BF16) for h in (H, kv, kv))
        out, lse, dout, got = step(gdn_lib, 2 * q, k, v, None)
        want = formula(2 * q, k, v, out, lse, dout, d ** -0.5)
        for (grad, _), name in zip(want, ("dq", "dk", "dv")):
            off = (got[name].double() - grad).norm()
            assert off <= 1.125 * (grad.to(BF16).double() - grad).norm(), (n, name)


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("T,H,kv", [(300, 2, 1), (4096, 16, 16)])      # jobs from the sequences; a list
def test_malformed_sequences_write_nothing(gdn_lib, T, H, kv, which):
    """Through the C call, whose results are the caller's; the call behind it finds its scratch and
    its inputs as they belong."""
    gdn = gdn_lib
    d, half = 64, T // 2
    q, k, v = inputs(T, T, H, kv, d)
    good = cu([half, T - half])
    out, lse, dout, want = step(gdn, q, k, v, good)
    for bad in ([0, T + 1, T], [1, half, T], [0, half, T - 1], [0, -1, T]):
        wrong = torch.tensor(bad, dtype=torch.int32, device="cuda")
        got = [torch.full_like(t, 7) for t in (q, k, v)]
        c = (wrong, good) if which == "q" else (good, wrong)
        gdn._call("gdn_attention_prefill_backward", q.get_device(), None,
                  *(t.data_ptr() for t in (q, k, v, out, lse, dout, *c)), d ** -0.5,
                  *(t.data_ptr() for t in got), 2, T, T, H, kv, d, H * d, kv * d, kv * d)
        again = gdn.attention_prefill_backward(q, k, v, out, lse, dout, good)
        assert gdn.device_status() == BAD_SEQLENS
        assert all((t == 7).all() for t in got)
        assert all(torch.equal(want[n], again[n]) for n in want)
