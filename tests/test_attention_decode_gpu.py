"""Attention of one new token over the paged cache against the formula in 64 bits.

Tolerance, element by element, with A = sum_j p_j |v_j| (p normalised): the result's rounding
2^-8 |o|; each probability's (8 bits: times the value's scale) rounding to bf16, 2^-8 A; the
exponents' errors, those of a sum of d fp32 products and of 2^x, under 2^-16 (1 + max |s|) of A
each for d <= 128 (d 2^-24 sum |q k| scale <= 2^-16 for |q| |k| scale <= 2; more is counted by
max |s| + the norms' product)."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
BAD = 9


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(gdn, lengths, kv, d, page, dtype, seed=0, layers=1, spare=3, max_pages=None):
    """A cache with these lengths on scattered pages and random contents."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    width = max_pages or max(1, max(need))
    pages = sum(need) + spare
    cache = gdn.kv_cache(layers, pages, kv, len(lengths), width, page, d, dtype)
    for pool, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = torch.randn(pool.shape, generator=g, device="cuda").to(BF16)
        if dtype == FP8:
            q, s = gdn.quantize_fp8(x)
            pool.view(torch.uint8).copy_(q.view(torch.uint8))
            scale.copy_(s[..., 0])
        else:
            pool.copy_(x)
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    table, at = torch.full((len(lengths), width), -1, dtype=torch.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    cache.table.copy_(table)
    cache.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    return cache


def row_of(cache, layer, r, n):
    page = cache.k.shape[3]
    ids = cache.table[r, :-(-n // page)].long()
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = (t.view(torch.uint8)[layer][ids].view(FP8) if t.dtype == FP8 else t[layer][ids]).double()
        if s is not None:
            x = x * s[layer][ids].double()[..., None]
        out.append(x.transpose(0, 1).flatten(1, 2)[:, :n])
    return out


def verify(q, cache, out, layer=0, scale=None, rows=None):
    H, d = q.shape[1:]
    kv = cache.k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    for r in range(q.shape[0]) if rows is None else rows:
        n = int(cache.lengths[r])
        if n == 0:
            assert (out[r] == 0).all()
            continue
        k, v = row_of(cache, layer, r, n)
        qr = q[r].double().view(kv, H // kv, d)
        s = scale * qr @ k.transpose(1, 2)
        p = torch.softmax(s, -1)
        o, A = p @ v, p @ v.abs()
        size = scale * qr.norm(dim=-1, keepdim=True) * k.norm(dim=-1).amax(-1)[:, None, None]
        tol = 2.0 ** -8 * 1.01 * (o.abs() + A) + A * 2.0 ** -16 * (1 + size)
        off = (out[r].double().view_as(o) - o).abs()
        assert (off <= tol).all(), (r, n, float((off - tol).max()))


EDGES = [0, 1, 2, 15, 16, 17, 0, 31, 33, 63, 64, 65, 127, 128, 129, 191, 193, 255, 256, 257, 1000]


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,kv,group", [(16, 2, 4), (32, 1, 5), (64, 4, 1), (128, 3, 16),
                                           (256, 1, 17), (16, 1, 128)])
def test_lengths_pages_and_groups(gdn_lib, dtype, d, page, kv, group):
    gdn = gdn_lib
    cache = filled(gdn, EDGES, kv, d, page, dtype, layers=2)
    q = (2 * torch.randn(len(EDGES), kv * group, d, device="cuda")).to(BF16)
    for layer in (0, 1):
        verify(q, cache, gdn.attention_decode_step(q, cache, layer), layer)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("rows,most", [(1, 1), (1, 5000), (3, 40000), (300, 700), (1100, 90)])
def test_splits(gdn_lib, dtype, rows, most):
    """One row over the whole GPU, many short ones, rows cut by the CTAs' parts."""
    gdn, rng = gdn_lib, random.Random(most)
    lengths = [most] + [rng.randint(0, most) for _ in range(rows - 1)]
    cache = filled(gdn, lengths, 2, 128, 64, dtype)
    q = torch.randn(rows, 6, 128, device="cuda").to(BF16)
    out = gdn.attention_decode_step(q, cache)
    verify(q, cache, out, rows=range(0, rows, max(1, rows // 50)))
    for _ in range(3):      # the same bits whatever runs first
        assert torch.equal(out, gdn.attention_decode_step(q, cache))
    ws = torch.empty(gdn.attention_decode_step_workspace_size(rows, 6, 2, 128), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(255)
    assert torch.equal(out, gdn.attention_decode_step(q, cache, workspace=ws))


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_sharp_scores_and_scales(gdn_lib, dtype):
    """Scores far apart (one key takes all), a large and a small scale, keys of every size."""
    gdn = gdn_lib
    cache = filled(gdn, [700, 64, 3], 1, 128, 32, dtype)
    q = (30 * torch.randn(3, 2, 128, device="cuda")).to(BF16)
    for scale in (None, 1.0, 1e-4):
        verify(q, cache, gdn.attention_decode_step(q, cache, scale=scale), scale=scale)
    if dtype == FP8:
        cache.v_scale.mul_(torch.exp2(torch.randint(-40, 40, cache.v_scale.shape, device="cuda").float()))
        verify(q, cache, gdn.attention_decode_step(q, cache))
    zero = torch.zeros_like(q)
    verify(zero, cache, gdn.attention_decode_step(zero, cache))


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_nothing_outside_a_row_is_read(gdn_lib, dtype):
    """NaN behind the last token, on free pages and in other rows changes nothing; in a row's own
    values it stays in the row."""
    gdn = gdn_lib
    lengths = [100, 65, 1, 130]
    cache = filled(gdn, lengths, 2, 64, 64, dtype)
    q = torch.randn(4, 4, 64, device="cuda").to(BF16)
    out = gdn.attention_decode_step(q, cache)
    used = torch.zeros(cache.k.shape[1], 64, dtype=torch.bool, device="cuda")
    for r, n in enumerate(lengths):
        for i in range(n):
            used[int(cache.table[r, i // 64]), i % 64] = True
    for t in (cache.k, cache.v):
        nan = 0x7f if dtype == FP8 else 0x7fff
        raw = t.view(torch.uint8 if dtype == FP8 else torch.int16)
        raw.masked_fill_(~used[None, :, None, :, None], nan)
    for t in (cache.k_scale, cache.v_scale):
        if t is not None:
            t.masked_fill_(~used[None, :, None, :], float("nan"))
    assert torch.equal(out, gdn.attention_decode_step(q, cache))
    page = int(cache.table[3, 1])
    if dtype == FP8:
        cache.v_scale[0, page, 1, 3] = float("nan")
    else:
        cache.v[0, page, 1, 3, 9] = float("nan")
    got = gdn.attention_decode_step(q, cache)
    assert torch.equal(got[:3], out[:3]) and torch.equal(got[3, :2], out[3, :2])
    assert got[3, 2:].isnan().any()
    assert gdn.device_status() == 0


def test_bad_lengths_and_pages_are_flagged(gdn_lib):
    gdn = gdn_lib
    lengths = [100, 65, 20, 130]
    cache = filled(gdn, lengths, 2, 64, 16, BF16)
    q = torch.randn(4, 4, 64, device="cuda").to(BF16)
    out = gdn.attention_decode_step(q, cache)
    cache.lengths[0], cache.lengths[2] = -5, cache.table.shape[1] * 16 + 1
    got = gdn.attention_decode_step(q, cache)
    assert gdn.device_status() == BAD
    assert (got[0] == 0).all() and (got[2] == 0).all()
    assert torch.equal(got[1], out[1]) and torch.equal(got[3], out[3])
    cache.table[1, 2], cache.table[1, 3] = -1, cache.k.shape[1]
    got = gdn.attention_decode_step(q, cache)
    assert gdn.device_status() == BAD
    assert torch.equal(got[3], out[3]) and got.isfinite().all()


def test_in_a_graph_beside_another(gdn_lib):
    """Two captured graphs with scratch of their own, replayed in turn and side by side; the rows
    grow between replays."""
    gdn = gdn_lib
    streams, graphs, parts = [torch.cuda.Stream() for _ in range(2)], [], []
    for i, st in enumerate(streams):
        cache = filled(gdn, [50 + i, 900, 0], 2, 128, 16, BF16, seed=i, max_pages=64, spare=50)
        gdn_refs = torch.zeros_like(cache.refs)
        gdn_refs[cache.table[cache.table >= 0].long()] = 1
        cache.refs.copy_(gdn_refs)
        q = torch.randn(3, 8, 128, device="cuda").to(BF16)
        one = ints([1, 1, 1])
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            gdn.attention_decode_step(q, cache)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                start = gdn.cache_reserve(cache, one)
                gdn.cache_append(cache, q[:, :2], q[:, 2:4], start)
                out = gdn.attention_decode_step(q, cache)
        graphs.append(graph)
        parts.append((q, cache, out))
    for _ in range(20):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for i, (q, cache, out) in enumerate(parts):
        assert cache.lengths.tolist() == [70 + i, 920, 20]
        verify(q, cache, out)
    assert gdn.device_status() == 0


def test_a_pool_of_more_than_2_31_elements(gdn_lib):
    gdn = gdn_lib
    pages = (2 ** 31 + 2 ** 24) // (4 * 256 * 128)
    cache = gdn.kv_cache(1, pages, 4, 2, 8, 256, 128)
    cache.table[0, :4] = ints([pages - 1, 0, pages - 2, pages - 3])
    cache.table[1, :1] = ints([pages - 4])
    cache.lengths.copy_(ints([1000, 77]))
    for t in (cache.k, cache.v):
        t[0, pages - 4:] = torch.randn(4, 4, 256, 128, device="cuda").to(BF16)
        t[0, 0] = torch.randn(4, 256, 128, device="cuda").to(BF16)
    q = torch.randn(2, 8, 128, device="cuda").to(BF16)
    verify(q, cache, gdn.attention_decode_step(q, cache))
