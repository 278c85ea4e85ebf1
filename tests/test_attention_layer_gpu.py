"""The attention layer's calls together, as a model makes them: packed prompts and single tokens
through the paged cache give the outputs of a prefill of the longer prompts; forked rows go their
own ways; a captured decoding step replays; the direct calls answer and agree with the general
path; calls on a device or stream of their own."""
import os
import sys

import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cu_of(lens):
    return ints([sum(lens[:i]) for i in range(len(lens) + 1)])


def test_the_example_runs(gdn_lib, capsys):
    import attention_layer
    attention_layer.main()
    assert "gradient norms" in capsys.readouterr().out


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_tokens_after_prompts_match_the_longer_prompts(gdn_lib, dtype):
    """Both paths round the probabilities (2^-8 of sum p |v| each) and the result; in 8 bits a key
    and a value are off by 2^-4 of themselves at most, so the outputs are compared in norm: bf16
    within 2^-7, 8 bits within 2^-3 (scores of unit size)."""
    kv, G, d, rows = 2, 3, 64, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    lens, more = [70, 1, 200, 64, 33], 3
    full = [n + more for n in lens]
    x = [[torch.randn(n, h, d, generator=g, device="cuda").to(BF16) for h in (kv * G, kv, kv)]
         for n in full]
    cache = gdn.kv_cache(1, 40, kv, rows, 8, 32, d, dtype)
    start = gdn.cache_reserve(cache, ints(lens))
    gdn.cache_append(cache, *(torch.cat([t[j][:n] for t, n in zip(x, lens)]) for j in (1, 2)), start,
                     cu_of(lens))
    one = ints([1] * rows)
    outs = []
    for t in range(more):
        q, k, v = (torch.stack([r[j][n + t] for r, n in zip(x, lens)]) for j in range(3))
        gdn.cache_append(cache, k, v, gdn.cache_reserve(cache, one))
        outs.append(gdn.attention_decode_step(q, cache))
    want, _ = gdn.attention_prefill(*(torch.cat([r[j] for r in x]) for j in range(3)), cu_of(full))
    ends = [sum(full[:i + 1]) for i in range(rows)]
    for t in range(more):
        ref = torch.stack([want[e - more + t] for e in ends]).float()
        off = (outs[t].float() - ref).norm() / ref.norm()
        assert off <= (2.0 ** -7 if dtype == BF16 else 2.0 ** -3), float(off)
    assert gdn.device_status() == 0


def test_prompts_in_pieces_match_the_whole(gdn_lib):
    """A prompt whose second half attends with the first as its stored context; its gradients add up
    to the whole's."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n, cut, H, kv, d = 300, 173, 6, 2, 128
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(BF16) for h in (H, kv, kv))
    dout = torch.randn(n, H, d, generator=g, device="cuda").to(BF16)
    out, lse = gdn.attention_prefill(q, k, v)
    a = gdn.attention_prefill(q[:cut], k[:cut], v[:cut])
    b = gdn.attention_prefill(q[cut:], k, v)
    pieces, sums = torch.cat([a[0], b[0]]), torch.cat([a[1], b[1]])
    assert (pieces.float() - out.float()).norm() <= 2.0 ** -7 * out.float().norm()
    assert (sums - lse).abs().max() <= 2.0 ** -14 * (1 + lse.abs().max())
    whole = gdn.attention_prefill_backward(q, k, v, out, lse, dout)
    ga = gdn.attention_prefill_backward(q[:cut], k[:cut], v[:cut], out[:cut].contiguous(),
                                        lse[:cut].contiguous(), dout[:cut].contiguous())
    gb = gdn.attention_prefill_backward(q[cut:], k, v, out[cut:].contiguous(), lse[cut:].contiguous(),
                                        dout[cut:].contiguous())
    dq = torch.cat([ga["dq"], gb["dq"]]).float()
    assert (dq - whole["dq"].float()).norm() <= 2.0 ** -6 * dq.norm()
    for name in ("dk", "dv"):
        s = gb[name].float()
        s[:cut] += ga[name].float()
        assert (s - whole[name].float()).norm() <= 2.0 ** -6 * s.norm(), name


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_a_next_turn_behind_the_stored_context(gdn_lib, dtype):
    """New tokens of rows that hold a context: appended to the pages, and attended with the gathered
    context as their keys.  In bf16 these are the bits that the whole prompts' tails have as
    queries of their own; in 8 bits the keys and values are off by 2^-4 of themselves at most."""
    kv, G, d = 2, 3, 64
    g = torch.Generator(device="cuda").manual_seed(13)
    lens, new = [70, 0, 200, 33], [5, 9, 0, 64]
    full = [a + b for a, b in zip(lens, new)]
    x = [[torch.randn(n, h, d, generator=g, device="cuda").to(BF16) for h in (kv * G, kv, kv)]
         for n in full]
    cache = gdn.kv_cache(2, 40, kv, 4, 8, 32, d, dtype)
    for counts, part in ((lens, lambda t, n: t[:n]), (new, lambda t, n: t[n:])):
        start = gdn.cache_reserve(cache, ints(counts))
        gdn.cache_append(cache, *(torch.cat([part(t[j], n) for t, n in zip(x, lens)]) for j in (1, 2)),
                         start, cu_of(counts), 1)
    k, v = gdn.cache_gather(cache, cu_of(full), sum(full), 1)
    q = torch.cat([t[0][n:] for t, n in zip(x, lens)])
    got, lse = gdn.attention_prefill(q, k, v, cu_of(new), cu_of(full))
    want, sums = gdn.attention_prefill(q, *(torch.cat([t[j] for t in x]) for j in (1, 2)), cu_of(new),
                                       cu_of(full))
    if dtype == BF16:
        assert torch.equal(got, want) and torch.equal(lse, sums)
    else:
        assert (got.float() - want.float()).norm() <= 2.0 ** -3 * want.float().norm()
    assert gdn.device_status() == 0


def test_a_captured_decoding_step(gdn_lib):
    """Reserve, append and attention of two layers in one graph, replayed with new inputs; the same
    from calls outside it, bit for bit."""
    kv, d, rows, layers = 2, 128, 6, 2
    g = torch.Generator(device="cuda").manual_seed(7)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    lens = [5, 64, 0, 127, 300, 31]
    caches = [gdn.kv_cache(layers, 60, kv, rows, 12, 32, d) for _ in range(2)]
    first = [new(sum(lens), kv, d) for _ in range(2)]
    for c in caches:
        start = gdn.cache_reserve(c, ints(lens))
        for layer in range(layers):
            gdn.cache_append(c, first[0], first[1], start, cu_of(lens), layer)
    counts = ints([1, 1, 1, 1, 0, 1])
    q, k, v = new(layers, rows, 8, d), new(layers, rows, kv, d), new(layers, rows, kv, d)

    def step(c):
        start = gdn.cache_reserve(c, counts)
        outs = []
        for layer in range(layers):
            gdn.cache_append(c, k[layer], v[layer], start, layer=layer)
            outs.append(gdn.attention_decode_step(q[layer], c, layer))
        return outs

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    lengths = caches[0].lengths.clone()
    with torch.cuda.graph(graph):
        got = step(caches[0])
    assert torch.equal(caches[0].lengths, lengths)       # captured, not run
    for _ in range(40):
        for t in (q, k, v):
            t.copy_(new(*t.shape))
        graph.replay()
        want = step(caches[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert caches[0].lengths.tolist() == [45, 104, 40, 167, 300, 71]
    assert gdn.device_status() == 0


def arguments():
    g = torch.Generator(device="cuda").manual_seed(11)
    q, k, v = (torch.randn(50, h, 64, generator=g, device="cuda").to(BF16) for h in (4, 2, 2))
    c = cu_of([20, 30])
    out, lse = gdn.attention_prefill(q, k, v, c)
    cache = gdn.kv_cache(2, 9, 2, 3, 4, 16, 64)
    start = gdn.cache_reserve(cache, ints([20, 1, 0]))
    gdn.cache_append(cache, k[:21], v[:21], start, cu_of([20, 1, 0]), 1)
    return q, k, v, c, out, lse, cache


@pytest.mark.parametrize("name", ["attention_prefill", "attention_prefill_backward",
                                  "attention_decode_step", "cache_reserve", "cache_append", "cache_gather", "cache_free",
                                  "cache_fork", "cache_compact"])
def test_the_direct_call_answers(gdn_lib, name, monkeypatch):
    """Each direct call takes ordinary arguments itself, with the general path's bits."""
    def once():
        q, k, v, c, out, lse, cache = arguments()
        into = gdn.kv_cache(2, 5, 2, 3, 4, 16, 64)
        calls = {
            "attention_prefill": ((q, k, v, c, None, None), lambda: gdn.attention_prefill(q, k, v, c)),
            "attention_prefill_backward": (
                (q, k, v, c, None, None, out, lse, q),
                lambda: gdn.attention_prefill_backward(q, k, v, out, lse, q, c).values()),
            "attention_decode_step": ((cache.address, cache.index, q[:3], 1, None),
                                      lambda: gdn.attention_decode_step(q[:3], cache, 1)),
            "cache_reserve": ((cache.address, cache.index, ints([1, 2, 3])),
                              lambda: gdn.cache_reserve(cache, ints([1, 2, 3]))),
            "cache_append": ((cache.address, cache.index, k[:3], v[:3], ints([19, 0, -1]), None, 1),
                             lambda: gdn.cache_append(cache, k[:3], v[:3], ints([19, 0, -1]), layer=1)),
            "cache_gather": ((cache.address, cache.index, cu_of([20, 1, 0]), 21, 1),
                             lambda: gdn.cache_gather(cache, cu_of([20, 1, 0]), 21, 1)),
            "cache_free": ((cache.address, cache.index, ints([1])), lambda: gdn.cache_free(cache, ints([1]))),
            "cache_fork": ((cache.address, cache.index, ints([0]), ints([2])),
                           lambda: gdn.cache_fork(cache, ints([0]), ints([2]))),
            "cache_compact": ((cache.address, cache.index, into.address, into.index),
                              lambda: gdn.cache_compact(cache, into)),
        }
        return calls[name], cache, into

    def state(result, cache, into):
        flat = [] if isinstance(result, (bool, type(None), gdn.KVCache)) else (
            [result] if isinstance(result, torch.Tensor) else list(result))
        return flat + [t for x in (cache, into) for t in (x.k, x.v, x.table, x.lengths, x.refs)]

    (args, _), cache, into = once()
    before = gdn.kernel_launches()
    got = getattr(gdn._direct, name)(*args)
    assert got is not None and gdn.kernel_launches() > before
    got = state(got, cache, into)
    monkeypatch.setattr(gdn, "_direct", gdn._Declines())
    (_, public), cache, into = once()
    want = state(public(), cache, into)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a, b)


def test_outputs_of_the_caller_and_other_streams(gdn_lib):
    """out=, lse=, start=, stream=: the results of the plain calls; work on another stream waits
    for nothing but it."""
    q, k, v, c, out, lse, cache = arguments()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, s = torch.empty_like(out), torch.empty_like(lse)
    gdn.attention_prefill(q, k, v, c, out=o, lse=s, stream=side)
    grads = gdn.attention_prefill_backward(q, k, v, o, s, q, c, stream=side)
    d = torch.empty_like(q[:3])
    gdn.attention_decode_step(q[:3], cache, 1, out=d, stream=side)
    start = torch.empty(3, dtype=torch.int32, device="cuda")
    counts = ints([1, 0, 2])
    side.wait_stream(torch.cuda.current_stream())
    gdn.cache_reserve(cache, counts, start=start, stream=side)
    side.synchronize()
    assert torch.equal(o, out) and torch.equal(s, lse) and start.tolist() == [20, 1, 0]
    assert torch.equal(d, gdn.attention_decode_step(q[:3], arguments()[6], 1))
    want = gdn.attention_prefill_backward(q, k, v, out, lse, q, c)
    assert all(torch.equal(want[n], grads[n]) for n in want)


def test_the_examples_gradients(gdn_lib):
    """Of the attention between the example's projections, against autograd of the formula in 64
    bits: probabilities and dS are rounded to bf16 (2^-8), as are the results, so 2^-6 in norm."""
    import attention_layer
    layer = attention_layer.AttentionLayer(256, heads=4, kv_heads=2)
    g = torch.Generator(device="cuda").manual_seed(9)
    n = 150
    x = torch.randn(n, 256, generator=g, device="cuda").to(BF16)
    dout = torch.randn(n, 4, 128, generator=g, device="cuda").to(BF16)
    _, got = layer.train_core(x, ints([0, n]), dout)
    q, k, v = (t.double().transpose(0, 1).requires_grad_() for t in layer.project(x, None)[:3])
    s = q @ k.repeat_interleave(2, 0).transpose(1, 2) * 128 ** -0.5
    s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -float("inf"))
    o = s.softmax(-1) @ v.repeat_interleave(2, 0)
    o.backward(dout.double().transpose(0, 1))
    for t, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        want = t.grad.transpose(0, 1)
        assert (got[name].double() - want).norm() <= 2.0 ** -6 * want.norm(), name
