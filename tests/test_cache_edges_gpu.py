"""What the attention cache's calls leave behind where something is wrong: defined contents, and a
cache that goes on."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
FULL, BAD_SEQLENS, BAD = 8, 6, 9


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(lens):
    return ints([sum(lens[:i]) for i in range(len(lens) + 1)])


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("d,kv", [(64, 3), (128, 2)])
def test_gather_of_what_a_row_does_not_hold(gdn_lib, dtype, d, kv):
    """Zeros, also where the memory held something; what no sequence has is left; the rest arrives."""
    gdn = gdn_lib
    lens, more = [20, 3, 0, 17], [0, 40, 0, 1]
    cache = gdn.kv_cache(1, 6, kv, 4, 4, 16, d, dtype)
    x = torch.randn(sum(lens), kv, d, device="cuda").to(BF16)
    gdn.cache_append(cache, x, x, gdn.cache_reserve(cache, ints(lens)), cu_of(lens))
    start = gdn.cache_reserve(cache, ints(more))           # two pages are left, row 1 wants three
    assert start.tolist() == [20, -1, 0, 17] and gdn.device_status() == FULL
    y = torch.randn(sum(more), kv, d, device="cuda").to(BF16)
    gdn.cache_append(cache, y, y, start, cu_of(more))
    assert gdn.device_status() == 0
    full = [a + b for a, b in zip(lens, more)]
    held = [20, 3, 0, 18]
    want = gdn.cache_gather(cache, cu_of(held), sum(held))
    assert gdn.device_status() == 0
    room = [torch.full((sum(full) + 5, kv, d), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
    gdn._call("gdn_cache_gather", cache.index, None, cache.address, 0, cu_of(full).data_ptr(),
              sum(full) + 5, *(t.data_ptr() for t in room))
    assert gdn.device_status() == BAD_SEQLENS
    for t, w in zip(room, want):
        assert (t[sum(full):] == 7).all()                  # behind the last sequence
        for a, n, b, m in zip(cu_of(full).tolist(), full, cu_of(held).tolist(), held):
            assert torch.equal(t[a:a + m], w[b:b + m]) and (t[a + m:a + n] == 0).all()
    # the binding's own results, in memory that has just held something
    room = [torch.full((sum(full), kv, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2)]
    del room
    k, v = gdn.cache_gather(cache, cu_of(full), sum(full))
    assert gdn.device_status() == BAD_SEQLENS
    assert (k[23:60] == 0).all() and (v[23:60] == 0).all()
    cache.table[0, 1] = 6
    k, v = gdn.cache_gather(cache, cu_of(held), sum(held))
    assert gdn.device_status() == BAD
    assert torch.equal(k[:16], want[0][:16]) and torch.equal(v[20:], want[1][20:])
    assert (k[16:20] == 0).all() and (v[16:20] == 0).all()


@pytest.mark.parametrize("bad", [-1, -(2 ** 31), 65, 2 ** 31 - 1])
def test_freeing_a_row_of_bad_length_gives_its_pages_back(gdn_lib, bad):
    """Once, however often it is named; pages that another row shares lose one reference; the pool
    serves the next rows as if the length had been right."""
    gdn = gdn_lib
    cache = gdn.kv_cache(1, 9, 1, 4, 4, 16, 64)
    gdn.cache_reserve(cache, ints([50, 17, 0, 0]))
    gdn.cache_fork(cache, ints([0]), ints([2]))            # three pages shared, a fourth of its own
    assert cache.refs.tolist() == [2, 2, 2, 1, 1, 1, 1, 0, 0] and gdn.device_status() == 0
    cache.lengths[0] = bad
    gdn.cache_free(cache, ints([0, 3, 0, 0]))
    assert gdn.device_status() == BAD
    assert cache.lengths.tolist() == [0, 17, 50, 0]
    assert (cache.table[0] == -1).all()
    assert cache.refs.tolist() == [1, 1, 1, 0, 1, 1, 1, 0, 0]
    gdn.cache_free(cache, ints([0, 2]))
    assert gdn.device_status() == 0
    assert cache.refs.tolist() == [0, 0, 0, 0, 1, 1, 0, 0, 0]
    assert gdn.cache_reserve(cache, ints([64, 0, 0, 0])).tolist() == [0, 17, 0, 0]
    assert cache.table[0].tolist() == [0, 1, 2, 3] and gdn.device_status() == 0


@pytest.mark.parametrize("n", [8, 1030])
@pytest.mark.parametrize("bad", [-1, -3, -8, -(2 ** 31)])
def test_fork_with_lengths_below_zero(gdn_lib, bad, n):
    """Of a target: it is not empty, the pair is skipped and the row left as it is.  Of a source:
    the target stays empty.  Both are flagged, whatever the number of pairs."""
    gdn = gdn_lib
    rows = n + 2
    for which in ("target", "source"):
        cache = gdn.kv_cache(1, n + 8, 1, rows, 3, 16, 64)
        gdn.cache_reserve(cache, ints([20, 33] + [0] * n))
        # (a target whose length is the mark of its own pair, where there is such a pair)
        at = n + bad if 0 <= n + bad < n else n // 2
        broken = 2 + at if which == "target" else 1
        if which == "target":
            cache.table[broken, 0] = 1                     # (what it still holds)
        cache.lengths[broken] = bad
        src = [0 if which == "target" else i % 2 for i in range(n)]
        gdn.cache_fork(cache, ints(src), ints(list(range(2, rows))))
        assert gdn.device_status() == BAD
        lengths, first = cache.lengths.tolist(), cache.table[:, 0].tolist()
        for i in range(n):
            skipped = 2 + i == broken or src[i] == 1
            assert lengths[2 + i] == (bad if 2 + i == broken else 0 if skipped else 20), i
            assert first[2 + i] == (1 if 2 + i == broken else -1 if skipped else 0), i
        made = sum(s == 0 for s in src) - (which == "target")
        assert cache.refs[0] == 1 + made and int(cache.refs.clamp(max=1).sum()) == 5 + made


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (128, 64), (64, 128), (128, 256)])
def test_decoding_over_a_page_that_is_none(gdn_lib, dtype, d, page):
    """Its keys and values are zeros, bit for bit what a page of zeros gives, whatever the pool's
    pages hold; other rows do not change."""
    gdn = gdn_lib
    lens = [5 * page + 3, 40, 3 * page, 1]
    g = torch.Generator(device="cuda").manual_seed(page)
    cache = gdn.kv_cache(1, 5 + sum(-(-n // page) for n in lens), 2, 4, 6, page, d, dtype)
    x = [torch.randn(sum(lens), 2, d, generator=g, device="cuda").to(BF16) for _ in range(2)]
    gdn.cache_append(cache, *x, gdn.cache_reserve(cache, ints(lens)), cu_of(lens))
    q = torch.randn(4, 6, d, generator=g, device="cuda").to(BF16)
    whole = gdn.attention_decode_step(q, cache)
    pages = cache.k.shape[1]
    free = int((cache.refs == 0).nonzero()[-1])
    assert (cache.k[0, free].float() == 0).all() and (cache.v[0, free].float() == 0).all()
    places = [[(0, 0)], [(0, 5)], [(0, 1), (0, 2), (2, 2)], [(2, i) for i in range(3)], [(3, 0)]]
    table = cache.table.clone()
    for at in places:
        for r, i in at:
            cache.table[r, i] = free
        want = gdn.attention_decode_step(q, cache)
        assert gdn.device_status() == 0
        for number in (-1, pages, 2 ** 31 - 1, -(2 ** 31)):
            for r, i in at:
                cache.table[r, i] = number
            # what the pages that are none might be taken for
            pools = [t.view(torch.uint8) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)
                     if t is not None]
            kept = [t.clone() for t in pools]
            used = set(cache.table.flatten().tolist()) | {free}
            for t in pools:
                t[0, [p for p in range(pages) if p not in used]] = 0x7f
            got = gdn.attention_decode_step(q, cache)
            assert gdn.device_status() == BAD
            assert torch.equal(got, want), (at, number)
            for r in set(range(4)) - {r for r, _ in at}:
                assert torch.equal(got[r], whole[r])
            for t, was in zip(pools, kept):
                t.copy_(was)
        cache.table.copy_(table)


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("number", [-1, 8])
def test_fork_of_a_last_page_that_is_none(gdn_lib, dtype, number):
    """The copy's own page holds zeros there, not what its last owner left; nothing else changes."""
    gdn = gdn_lib
    cache = gdn.kv_cache(2, 8, 3, 3, 4, 16, 64, dtype)
    pools = [t.view(torch.uint8) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    for t in pools:
        t.random_(0, 100)
    gdn.cache_reserve(cache, ints([21, 0, 5]))             # pages 0, 1; 2
    cache.table[0, 1] = number
    was = [t.clone() for t in pools]
    gdn.cache_fork(cache, ints([0, 2]), ints([1, 1]))
    assert gdn.device_status() == BAD
    assert cache.lengths.tolist() == [21, 21, 5] and cache.table[1].tolist() == [0, 3, -1, -1]
    assert cache.refs.tolist() == [2, 1, 1, 1, 0, 0, 0, 0]
    for t, w in zip(pools, was):
        width = t.shape[3] // 16 if t.dim() == 4 else 1    # (scales: four bytes a token)
        w[:, 3, :, :5 * width] = 0
        assert torch.equal(t, w)
