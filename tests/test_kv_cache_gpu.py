"""The attention cache's pages on the GPU: integers against the rules on plain lists, contents
bit for bit (8 bits: the codes and scales of quantize_fp8)."""
import random

import pytest
import torch

from kv_cache_model import Model

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
FULL, BAD_SEQLENS, BAD = 8, 6, 9


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(cache, model):
    assert cache.lengths.tolist() == model.lengths
    assert cache.refs.tolist() == model.refs
    assert cache.table.tolist() == model.table()


def make(gdn, model, layers=1, kv=2, d=64, dtype=BF16):
    return gdn.kv_cache(layers, len(model.refs), kv, len(model.rows), model.max_pages, model.page, d,
                        dtype)


def bits(t):
    return t.view(torch.uint8) if t.dtype == FP8 else t.view(torch.int16) if t.dtype == BF16 else t


def stored(cache, layer, row, n):
    """The first n tokens of a row as they lie in the pool: k, v (and scales)."""
    page = cache.k.shape[3]
    ids = cache.table[row, :-(-n // page)].long()
    out = []
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            x = bits(t)[layer, ids].transpose(1, 2)       # pages, page, heads, ..
            out.append(x.reshape(-1, *x.shape[2:])[:n])
    return out


def expected(gdn, x, dtype):
    if dtype == BF16:
        return bits(x), None
    q, s = gdn.quantize_fp8(x.contiguous())
    return bits(q), s[..., 0]


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("d,page,kv", [(64, 16, 1), (128, 64, 4), (128, 256, 3), (64, 32, 8)])
def test_a_serving_history(gdn_lib, dtype, d, page, kv):
    """Prompts, tokens, forks, freed rows and a compaction in one run; after it every row holds
    exactly what was appended to it."""
    gdn, rng = gdn_lib, random.Random(page + d)
    rows, layers = 9, 2
    model = Model(rows, 12, 60, page)
    cache = make(gdn, model, layers, kv, d, dtype)
    held = [[torch.empty(2, 0, kv, d, device="cuda", dtype=BF16) for _ in range(layers)]
            for _ in range(rows)]
    g = torch.Generator(device="cuda").manual_seed(page)

    def append(counts):
        start = gdn.cache_reserve(cache, ints(counts))
        assert start.tolist() == model.reserve(counts)
        assert all(s >= 0 for s in start.tolist())
        cu = ints([sum(counts[:i]) for i in range(rows + 1)])
        for layer in range(layers):
            # a slice of a packed projection: q | k | v
            x = (3 * torch.randn(sum(counts), 4 * kv * d, generator=g, device="cuda")).to(BF16)
            k, v = (x[:, i * kv * d:(i + 1) * kv * d].unflatten(1, (kv, d)) for i in (1, 2))
            gdn.cache_append(cache, k, v, start, cu, layer)
            for r, (a, b) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
                held[r][layer] = torch.cat([held[r][layer], torch.stack([k[a:b], v[a:b]])], 1)

    def verify():
        check(cache, model)
        for r in range(rows):
            for layer in range(layers):
                n = model.lengths[r]
                assert held[r][layer].shape[1] == n
                want = [expected(gdn, held[r][layer][i], dtype) for i in (0, 1)]
                want = [want[0][0], want[1][0]] + ([want[0][1], want[1][1]] if dtype == FP8 else [])
                for a, b in zip(stored(cache, layer, r, n), want):
                    assert torch.equal(a, b)

    append([1, page, page - 1, 0, page + 1, 2 * page + 5, 0, 0, 0])
    verify()
    for _ in range(3):
        append([rng.randint(0, 1) for _ in range(rows)])
    verify()
    gdn.cache_free(cache, ints([6, 7, 8, 3]))
    model.free([6, 7, 8, 3])
    for r in (6, 7, 8, 3):
        held[r] = [t[:, :0] for t in held[r]]
    src, dst = [5, 5, 1, 3], [7, 8, 6, 3]      # row 3 is empty: so is its copy of itself
    gdn.cache_fork(cache, ints(src), ints(dst))
    model.fork(src, dst)
    for a, b in zip(src, dst):
        held[b] = list(held[a])
    verify()
    append([1] * rows)                          # the copies go apart
    verify()
    gdn.cache_free(cache, ints([5]))            # the pages that the copies share stay
    model.free([5])
    held[5] = [t[:, :0] for t in held[5]]
    verify()
    room = sum(r > 0 for r in model.refs) + 3
    order = model.compact(room)
    into = gdn.kv_cache(layers, room, kv, rows, 14, page, d, dtype)
    before = {n: bits(getattr(cache, n)).clone() for n in ("k", "v", "table", "lengths", "refs")}
    for t in (into.k, into.v):
        bits(t).fill_(77)
    into.refs.fill_(5)
    assert gdn.cache_compact(cache, into) is into
    for n, t in before.items():
        assert torch.equal(bits(getattr(cache, n)), t)
    for t in (into.k, into.v):
        assert (bits(t)[:, len(order):] == 77).all()
    model.max_pages, cache = 14, into
    verify()
    append([2] * rows)
    verify()
    assert gdn.device_status() == 0


@pytest.mark.parametrize("rows,pages,max_pages", [(3, 7, 4), (1500, 2500, 3), (40, 9001, 300)])
def test_pages_are_taken_in_order_and_run_out(gdn_lib, rows, pages, max_pages):
    gdn, rng = gdn_lib, random.Random(rows)
    model = Model(rows, max_pages, pages, 16)
    cache = make(gdn, model, kv=1)
    short = False
    for step in range(6):
        most = 16 * max_pages // (2 if step < 3 else 1)
        counts = [rng.choice([0, 1, 16, rng.randint(0, most), -1 if step == 4 else 3])
                  for _ in range(rows)]
        want = model.reserve(counts)
        start = gdn.cache_reserve(cache, ints(counts))
        assert start.tolist() == want
        check(cache, model)
        failed = -1 in want
        short |= failed
        status = gdn.device_status()
        assert (status in (FULL, BAD)) == failed and (failed or status == 0)
        rows_out = rng.sample(range(rows), rows // 3)
        gdn.cache_free(cache, ints(rows_out))
        model.free(rows_out)
        check(cache, model)
    assert short


def test_free_twice_and_out_of_range(gdn_lib):
    gdn = gdn_lib
    model = Model(4, 4, 20, 16)
    cache = make(gdn, model)
    gdn.cache_reserve(cache, ints([40, 1, 64, 0]))
    model.reserve([40, 1, 64, 0])
    gdn.cache_free(cache, ints([2, 2, 0, 2, 3, 3]))
    model.free([2, 0, 3])
    check(cache, model)
    assert gdn.device_status() == 0
    gdn.cache_free(cache, ints([-1, 4, 1, 2 ** 31 - 1]))
    model.free([1])
    check(cache, model)
    assert gdn.device_status() == BAD
    gdn.cache_free(cache, ints([]))
    assert gdn.device_status() == 0


@pytest.mark.parametrize("n", [8, 1400])
def test_fork_skips_what_it_cannot_do(gdn_lib, n):
    """Rows outside the cache, rows that hold something, the same target twice (the first pair
    counts), a pool without a page left."""
    gdn, rng = gdn_lib, random.Random(n)
    rows = 2 * n
    model = Model(rows, 3, 3 * n, 16)
    cache = make(gdn, model, kv=1)
    counts = [rng.choice([0, 5, 16, 33, 48]) if r < n // 2 else 0 for r in range(rows)]
    counts[0], counts[1] = 20, 0
    gdn.cache_reserve(cache, ints(counts))
    model.reserve(counts)
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, device="cuda"))
    src = [rng.randint(0, n // 2) for _ in range(n)]
    dst = [rng.randint(n // 4, rows - 1) for _ in range(n)]
    src[:7], dst[:7] = [0, 1, -1, 0, rows, 2, 0], [rows - 1, rows - 1, 5, rows - 2, 6, rows, rows - 2]
    was = cache.k.clone(), cache.v.clone()
    gdn.cache_fork(cache, ints(src), ints(dst))
    copies = model.fork(src, dst)
    check(cache, model)
    assert gdn.device_status() in (BAD, FULL)
    for old, t in zip(was, (cache.k, cache.v)):
        for a, b, tail in copies:
            old[:, b, :, :tail] = old[:, a, :, :tail]
        assert torch.equal(bits(old), bits(t))


@pytest.mark.parametrize("n", [4, 1030])
def test_fork_of_a_row_with_a_bad_length(gdn_lib, n):
    """The pair is skipped and its target stays empty; the others are made."""
    gdn = gdn_lib
    cache = gdn.kv_cache(1, 8 + n, 1, 2 + n, 3, 16, 64)
    gdn.cache_reserve(cache, ints([20, 20] + [0] * n))
    cache.lengths[1] = 3 * 16 + 1
    src = [i % 2 for i in range(n)]
    gdn.cache_fork(cache, ints(src), ints(list(range(2, 2 + n))))
    assert gdn.device_status() == BAD
    assert cache.lengths[2:].tolist() == [0 if i else 20 for i in src]
    assert ((cache.table[2:, 0] >= 0).long().tolist() == [1 - i for i in src])


def test_fork_without_a_page_left(gdn_lib):
    gdn = gdn_lib
    model = Model(5, 3, 4, 16)
    cache = make(gdn, model)
    counts = [20, 16, 0, 0, 0]
    gdn.cache_reserve(cache, ints(counts))
    model.reserve(counts)
    # one page is left: the second pair gets none, the third needs none
    src, dst = [0, 0, 1], [2, 3, 4]
    gdn.cache_fork(cache, ints(src), ints(dst))
    model.fork(src, dst)
    check(cache, model)
    assert model.lengths == [20, 16, 20, 0, 16]
    assert gdn.device_status() == FULL
    gdn.cache_fork(cache, ints([]), ints([]))
    assert gdn.device_status() == 0


def test_compact_without_room_writes_nothing(gdn_lib):
    gdn = gdn_lib
    model = Model(2, 4, 9, 16)
    cache, into = make(gdn, model), gdn.kv_cache(1, 4, 2, 2, 4, 16, 64)
    gdn.cache_reserve(cache, ints([64, 16]))
    for t in (into.table, into.lengths, into.refs):
        t.fill_(3)
    gdn.cache_compact(cache, into)
    assert gdn.device_status() == FULL
    assert all((t == 3).all() for t in (into.table, into.lengths, into.refs))
    assert (into.k == 0).all()


def test_append_skips_bad_places(gdn_lib):
    """Rows that got no place, page numbers outside the pool, tokens outside their cu_seqlens."""
    gdn = gdn_lib
    model = Model(4, 2, 6, 16)
    cache = make(gdn, model)
    k = torch.randn(4, 2, 64, device="cuda").to(BF16)
    gdn.cache_reserve(cache, ints([1, 1, 1, 1]))
    cache.table[1, 0], cache.table[2, 0] = 6, -1
    gdn.cache_append(cache, k, k, ints([0, 0, 0, -1]))
    assert gdn.device_status() == BAD
    assert torch.equal(cache.k[0, 0, :, 0], k[0]) and cache.k.count_nonzero() == k[0].count_nonzero()
    cache.lengths.copy_(ints([33, 33, 32, 16]))
    gdn.cache_append(cache, k, k, ints([-7, 32, -1, 15]))      # behind the table, below -1
    assert gdn.device_status() == BAD
    assert torch.equal(cache.k[0, 3, :, 15], k[3])
    assert cache.k.count_nonzero() == k[0].count_nonzero() + k[3].count_nonzero()
    before = cache.k.clone()
    gdn.cache_append(cache, k, k, ints([33, 34, 40, 16]))      # not reserved: nothing, silently
    assert gdn.device_status() == 0 and torch.equal(before, cache.k)
    for cu in ([0, 1, 0, 1, 2], [5, 6, 7, 8, 9], [0, 0, 0, 0, 0], [0, -5, -5, -5, 0]):
        gdn.cache_append(cache, k, k, ints([-1, -1, -1, -1]), ints(cu))
        assert gdn.device_status() == BAD_SEQLENS
    assert torch.equal(before, cache.k)
    gdn.cache_append(cache, k[:0], k[:0], ints([0] * 4), ints([0] * 5))
    assert gdn.device_status() == 0


def test_eight_bit_extremes(gdn_lib):
    """Zeros, the type's largest and smallest numbers, an infinity and a NaN: the codes and scales
    are quantize_fp8's."""
    gdn = gdn_lib
    cache = gdn.kv_cache(1, 8, 1, 6, 1, 16, 128, FP8)
    x = torch.randn(6, 1, 128, device="cuda").to(BF16)
    x[0] = 0
    x[1, 0, ::2] = 3.3e38
    x[2] *= 2.0 ** -125
    x[3, 0, 5] = float("inf")
    x[4, 0, 7] = float("nan")
    start = gdn.cache_reserve(cache, ints([1] * 6))
    gdn.cache_append(cache, x, x, start)
    q, s = gdn.quantize_fp8(x)
    assert torch.equal(bits(cache.k)[0, :6, :, 0], bits(q))
    assert torch.equal(cache.v_scale[0, :6, :, 0].nan_to_num(7), s[..., 0].nan_to_num(7))


def test_on_another_stream_and_in_a_graph(gdn_lib):
    """A captured step (reserve, append) replayed continues the cache; a second cache's graph
    between the replays changes nothing."""
    gdn = gdn_lib
    models = [Model(5, 6, 40, 16) for _ in range(2)]
    caches = [make(gdn, m) for m in models]
    k = torch.randn(5, 2, 64, device="cuda").to(BF16)
    one = ints([1, 0, 1, 1, 1])
    graphs, starts, side = [], [], torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c, m in zip(caches, models):
            gdn.cache_append(c, k, k, gdn.cache_reserve(c, one))
            m.reserve(one.tolist())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                starts.append(gdn.cache_reserve(c, one))
                gdn.cache_append(c, k, k, starts[-1])
                gdn.cache_free(c, ints_of_row4)
                gdn.cache_fork(c, ints_of_row0, ints_of_row4)
            graphs.append(graph)
        for step in range(40):
            for graph, m, s in zip(graphs, models, starts):
                graph.replay()
                want = m.reserve(one.tolist())
                m.free([4])
                m.fork([0], [4])
                assert s.tolist() == want
        for c, m in zip(caches, models):
            check(c, m)
            for r in (0, 2, 3, 4):
                assert torch.equal(stored(c, 0, r, m.lengths[r])[0],
                                   bits(k[0 if r == 4 else r]).expand(m.lengths[r], 2, 64))
    assert gdn.device_status(side) == 0


@pytest.fixture(autouse=True)
def row_numbers(gdn_lib):
    global ints_of_row0, ints_of_row4
    ints_of_row0, ints_of_row4 = ints([0]), ints([4])
    torch.cuda.synchronize()


def test_a_pool_of_more_than_2_31_elements(gdn_lib):
    """Pages whose elements lie behind 2^31 and 2^32."""
    gdn = gdn_lib
    pages = (2 ** 32 + 2 ** 24) // (4 * 256 * 128)
    cache = gdn.kv_cache(1, pages, 4, 2, 40, 256, 128, FP8)
    first = pages - 40
    cache.refs[:first] = 1
    counts = [256 * 30 + 3, 256 * 5]
    start = gdn.cache_reserve(cache, ints(counts))
    assert start.tolist() == [0, 0] and cache.table[0, :31].tolist() == list(range(first, first + 31))
    x = torch.randn(sum(counts), 4, 128, device="cuda").to(BF16)
    gdn.cache_append(cache, x, x, start, ints([0, counts[0], sum(counts)]))
    q, s = gdn.quantize_fp8(x)
    for r, part in ((0, slice(0, counts[0])), (1, slice(counts[0], None))):
        got = stored(cache, 0, r, counts[r])
        assert torch.equal(got[1], bits(q)[part]) and torch.equal(got[2], s[part, :, 0])
    gdn.cache_free(cache, ints([1]))
    gdn.cache_fork(cache, ints([0]), ints([1]))
    assert torch.equal(stored(cache, 0, 1, counts[0])[0], bits(q)[:counts[0]])
    cache.refs[:first] = 0
    into = gdn.kv_cache(1, 64, 4, 2, 40, 256, 128, FP8)
    gdn.cache_compact(cache, into)
    assert torch.equal(stored(into, 0, 1, counts[0])[0], bits(q)[:counts[0]])
    assert gdn.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("d,page,kv", [(64, 16, 3), (128, 64, 2), (128, 256, 1)])
def test_gather(gdn_lib, dtype, d, page, kv):
    """The stored tokens in order; codes times their scales rounded to bf16; fewer than a row holds;
    what a row does not hold is flagged and left."""
    gdn = gdn_lib
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = [0, 1, 130, 16, 0, 257, 64]
    need = sum(-(-n // page) for n in lens)
    cache = gdn.kv_cache(2, need + 2, kv, len(lens), 20, page, d, dtype)
    x = [torch.randn(sum(lens), kv, d, generator=g, device="cuda").to(BF16) for _ in range(2)]
    starts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    gdn.cache_append(cache, *x, gdn.cache_reserve(cache, ints(lens)), ints(starts), 1)
    if dtype == FP8:
        x = [(c.float().unflatten(-1, (-1, d)) * s[..., None]).flatten(-2).to(BF16)
             for c, s in (gdn.quantize_fp8(t.reshape(-1, d)) for t in x)]
        x = [t.view(-1, kv, d) for t in x]
    for counts in (lens, [0, 1, 100, 0, 0, 256, 64], [0] * 6 + [3]):
        cu = [sum(counts[:i]) for i in range(len(counts) + 1)]
        at = [starts[r] + i for r, n in enumerate(counts) for i in range(n)]
        got = gdn.cache_gather(cache, ints(cu), cu[-1], 1)
        assert all(torch.equal(a, b[at]) for a, b in zip(got, x))
    none = gdn.cache_gather(cache, ints([0] * 8), 0, 1)
    assert none[0].shape == (0, kv, d) and gdn.device_status() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn.cache_gather(cache, ints(starts), starts[-1], 1, stream=side)
    side.synchronize()
    assert torch.equal(got[1], x[1])
    gdn.cache_gather(cache, ints([0, 0, 2, 2, 2, 2, 2, 2]), 2, 1)
    assert gdn.device_status() == 6
    gdn.cache_gather(cache, ints([0, 0, 1, 1, 1, 1, 1, 1]), 2, 1)
    assert gdn.device_status() == 6
    cache.table[1, 0] = need + 2
    gdn.cache_gather(cache, ints([0, 0, 1, 1, 1, 1, 1, 1]), 1, 1)
    assert gdn.device_status() == BAD
