"""The attention layers' calls and their cache refuse malformed host arguments before they touch
the GPU, at the C ABI (status codes) and in the Python binding.  CPU only: the C calls get fake
addresses and do not run where a CUDA device is visible."""
import ctypes

import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn
from test_abi import fake_addresses, lib  # noqa: F401  (fixture)

P = ctypes.c_void_p
SIZE_MAX = ctypes.c_size_t(-1).value
A = [P(0x100000000 * (i + 1)) for i in range(14)]
MIS = P(0x100000008)
BF16, E4M3 = 1, 2


@pytest.fixture(autouse=True)
def no_launch(request):
    if "lib" not in request.fixturenames:
        yield
        return
    library = request.getfixturevalue("lib")
    before = library.gdn_kernel_launches()
    yield
    assert library.gdn_kernel_launches() == before, "a host-argument test launched a kernel"


@fake_addresses
def test_prefill_refuses(lib):  # noqa: F811
    def f(q=A[0], k=A[1], v=A[2], cq=None, ck=None, scale=0.1, out=A[3], lse=A[4], n=2, tq=16, tk=16,
          h=8, kv=2, d=64, qs=512, ks=128, vs=128):
        return lib.gdn_attention_prefill(q, k, v, cq, ck, scale, out, lse, n, tq, tk, h, kv, d, qs, ks,
                                         vs, None)
    assert f(tq=0) == 0
    assert f(n=0) == 1 and f(tq=-1) == 1 and f(tk=-1) == 1 and f(h=0) == 1 and f(kv=0) == 1
    assert f(scale=0.0) == 1 and f(scale=-1.0) == 1 and f(scale=float("nan")) == 1
    assert f(scale=float("inf")) == 1
    assert f(q=None) == 1 and f(out=None) == 1 and f(lse=None) == 1 and f(k=None) == 1 and f(v=None) == 1
    assert f(cq=A[5]) == 1 and f(ck=A[5]) == 1                    # both or neither
    assert f(d=32) == 2 and f(d=256) == 2 and f(kv=3) == 2 and f(h=129, kv=1, qs=129 * 64, ks=64, vs=64) == 2
    assert f(n=1, tq=2 ** 31) == 2 and f(n=1, tk=2 ** 31) == 2 and f(n=2 ** 20, tq=2 ** 20) == 2
    assert f(qs=511) == 1 and f(ks=120) == 1 and f(vs=64) == 1    # narrower than the heads
    assert f(qs=516) == 3 and f(ks=132) == 3 and f(vs=129) == 3
    assert f(q=MIS) == 3 and f(k=MIS) == 3 and f(v=MIS) == 3 and f(out=P(A[3].value + 8)) == 3
    assert f(lse=P(A[4].value + 2)) == 3 and f(cq=P(A[5].value + 1), ck=A[6]) == 3
    assert f(out=A[0]) == 1 and f(lse=A[3]) == 1 and f(lse=A[1]) == 1
    assert f(out=P(A[0].value + 16)) == 1


@fake_addresses
def test_backward_refuses(lib):  # noqa: F811
    def f(q=A[0], k=A[1], v=A[2], out=A[3], lse=A[4], dout=A[5], cq=None, ck=None, scale=0.1, dq=A[6],
          dk=A[7], dv=A[8], n=2, tq=16, tk=16, h=8, kv=2, d=64, qs=512, ks=128, vs=128, ws=None, wb=None):
        args = (q, k, v, out, lse, dout, cq, ck, scale, dq, dk, dv, n, tq, tk, h, kv, d, qs, ks, vs)
        if wb is None:
            return lib.gdn_attention_prefill_backward(*args, None)
        return lib.gdn_attention_prefill_backward_ws(*args, ws, wb, None)
    assert f(tq=0, tk=0) == 0
    for name in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"):
        assert f(**{name: None}) == 1, name
    for name, at in (("q", 0), ("out", 3), ("dout", 5), ("dq", 6), ("dk", 7), ("dv", 8)):
        assert f(**{name: P(A[at].value + 8)}) == 3, name
    assert f(lse=P(A[4].value + 2)) == 3
    assert f(d=96) == 2 and f(kv=3) == 2 and f(scale=0.0) == 1 and f(cq=A[9]) == 1 and f(qs=500) == 1
    assert f(dq=A[0]) == 1 and f(dk=A[8]) == 1 and f(dv=A[3]) == 1 and f(dq=A[5]) == 1
    size = lib.gdn_attention_prefill_backward_workspace_size(2, 16, 16, 0, 8, 2, 64)
    assert 0 < size < SIZE_MAX
    assert f(ws=A[9], wb=size - 1) == 1 and f(ws=None, wb=size) == 1
    assert f(ws=P(A[9].value + 16), wb=size) == 3 and f(ws=A[0], wb=size) == 1
    for bad in ((0, 16, 16, 0, 8, 2, 64), (2, -1, 16, 0, 8, 2, 64), (2, 16, 16, 0, 8, 3, 64),
                (2, 16, 16, 0, 8, 2, 80), (2, 16, -1, 0, 8, 2, 64)):
        assert lib.gdn_attention_prefill_backward_workspace_size(*bad) == SIZE_MAX
    assert lib.gdn_attention_prefill_backward_workspace_size(2, 0, 16, 1, 8, 2, 64) == 0


def cache(at=0, **changes):
    fields = dict(k=A[at].value, v=A[at + 1].value, k_scale=None, v_scale=None, table=A[at + 2].value,
                  lengths=A[at + 3].value, refs=A[at + 4].value, layers=2, pages=8, kv_heads=2, page=16,
                  d=64, rows=4, max_pages=3, dtype=BF16)
    return gdn._CacheStruct(**dict(fields, **changes))


BAD_CACHES = [(dict(layers=0), 1), (dict(pages=0), 1), (dict(kv_heads=0), 1), (dict(rows=0), 1),
              (dict(max_pages=0), 1), (dict(dtype=0), 2), (dict(dtype=3), 2), (dict(page=24), 2),
              (dict(page=8), 2), (dict(page=512), 2), (dict(d=96), 2),
              (dict(max_pages=2 ** 27, page=16), 2), (dict(k=None), 1), (dict(v=None), 1),
              (dict(table=None), 1), (dict(lengths=None), 1), (dict(refs=None), 1),
              (dict(dtype=E4M3), 1), (dict(k_scale=A[9].value, v_scale=A[10].value), 1),
              (dict(dtype=E4M3, k_scale=A[9].value), 1), (dict(k=MIS.value), 3),
              (dict(refs=A[4].value + 4), 3), (dict(table=A[2].value + 2), 3)]


@fake_addresses
@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_a_malformed_cache_is_refused_by_every_call(lib, change, code):  # noqa: F811
    c, good = ctypes.byref(cache(**change)), ctypes.byref(cache(5))
    assert lib.gdn_cache_reserve(c, A[11], A[12], None) == code
    assert lib.gdn_cache_append(c, 0, A[11], A[12], A[13], None, 4, 128, 128, None) == code
    assert lib.gdn_cache_gather(c, 0, A[11], 4, A[12], A[13], None) == code
    assert lib.gdn_cache_free(c, A[11], 1, None) == code
    assert lib.gdn_cache_fork(c, A[11], A[12], 1, None) == code
    assert lib.gdn_cache_compact(c, good, None) == code
    assert lib.gdn_cache_compact(good, c, None) == code
    assert lib.gdn_attention_decode_step(A[11], c, 0, 4, 0.1, A[12], None) == code


@fake_addresses
def test_cache_calls_refuse(lib):  # noqa: F811
    c = ctypes.byref(cache())
    assert lib.gdn_cache_reserve(None, A[5], A[6], None) == 1
    assert lib.gdn_cache_reserve(c, None, A[6], None) == 1 and lib.gdn_cache_reserve(c, A[5], None, None) == 1
    assert lib.gdn_cache_reserve(c, P(A[5].value + 2), A[6], None) == 3
    assert lib.gdn_cache_reserve(c, A[5], A[5], None) == 1 and lib.gdn_cache_reserve(c, A[5], A[3], None) == 1
    assert lib.gdn_cache_reserve(c, A[4], A[6], None) == 1

    def append(layer=0, k=A[5], v=A[6], start=A[7], cu=None, n=4, ks=128, vs=128):
        return lib.gdn_cache_append(c, layer, k, v, start, cu, n, ks, vs, None)
    assert append(n=0, cu=A[8]) == 0
    assert append(layer=2) == 1 and append(layer=-1) == 1 and append(n=5) == 1 and append(n=-1, cu=A[8]) == 1
    assert append(k=None) == 1 and append(start=None) == 1 and append(ks=120) == 1
    assert append(ks=132) == 3 and append(k=P(A[5].value + 8)) == 3 and append(start=P(A[7].value + 1)) == 3
    assert append(k=A[0]) == 1 and append(start=A[3]) == 1

    def gather(layer=0, cu=A[5], n=4, k=A[6], v=A[7]):
        return lib.gdn_cache_gather(c, layer, cu, n, k, v, None)
    assert gather(n=0) == 0 and gather(n=0, k=None, v=None) == 0
    assert gather(layer=2) == 1 and gather(layer=-1) == 1 and gather(n=-1) == 1 and gather(n=2 ** 31) == 1
    assert gather(cu=None) == 1 and gather(k=None) == 1 and gather(v=None) == 1
    assert gather(cu=P(A[5].value + 2)) == 3 and gather(k=P(A[6].value + 8)) == 3
    assert gather(k=A[0]) == 1 and gather(v=A[6]) == 1 and gather(v=A[5]) == 1 and gather(k=A[3]) == 1
    assert lib.gdn_cache_free(c, None, 0, None) == 0
    assert lib.gdn_cache_free(c, A[5], -1, None) == 1 and lib.gdn_cache_free(c, None, 1, None) == 1
    assert lib.gdn_cache_free(c, P(A[5].value + 2), 1, None) == 3 and lib.gdn_cache_free(c, A[2], 1, None) == 1
    assert lib.gdn_cache_fork(c, None, None, 0, None) == 0
    assert lib.gdn_cache_fork(c, A[5], None, 1, None) == 1 and lib.gdn_cache_fork(c, A[5], A[6], -1, None) == 1
    assert lib.gdn_cache_fork(c, A[5], A[4], 1, None) == 1
    for change in (dict(layers=1), dict(kv_heads=1), dict(page=32), dict(d=128), dict(rows=5),
                   dict(max_pages=2)):
        assert lib.gdn_cache_compact(c, ctypes.byref(cache(5, **change)), None) == 1, change
    assert lib.gdn_cache_compact(c, c, None) == 1


@fake_addresses
def test_decode_refuses(lib):  # noqa: F811
    c = ctypes.byref(cache())

    def f(q=A[5], layer=0, h=4, scale=0.1, out=A[6], ws=None, wb=None):
        if wb is None:
            return lib.gdn_attention_decode_step(q, c, layer, h, scale, out, None)
        return lib.gdn_attention_decode_step_ws(q, c, layer, h, scale, out, ws, wb, None)
    assert f(q=None) == 1 and f(out=None) == 1 and f(layer=2) == 1 and f(layer=-1) == 1
    assert f(scale=0.0) == 1 and f(scale=float("nan")) == 1 and f(h=0) == 1
    assert f(h=3) == 2 and f(h=258) == 2
    assert f(q=P(A[5].value + 8)) == 3 and f(out=P(A[6].value + 8)) == 3
    assert f(out=A[5]) == 1 and f(out=A[0]) == 1
    size = lib.gdn_attention_decode_step_workspace_size(4, 4, 2, 64)
    assert 0 < size < SIZE_MAX
    assert f(ws=A[7], wb=size - 1) == 1 and f(ws=None, wb=size) == 1 and f(ws=A[0], wb=size) == 1
    assert f(ws=P(A[7].value + 64), wb=size) == 3
    for bad in ((0, 4, 2, 64), (4, 3, 2, 64), (4, 4, 2, 80), (4, 258, 2, 64)):
        assert lib.gdn_attention_decode_step_workspace_size(*bad) == SIZE_MAX


def cpu_cache(**changes):
    t = dict(k=torch.zeros(1, 8, 2, 16, 64, dtype=torch.bfloat16),
             v=torch.zeros(1, 8, 2, 16, 64, dtype=torch.bfloat16),
             table=torch.zeros(4, 3, dtype=torch.int32), lengths=torch.zeros(4, dtype=torch.int32),
             refs=torch.zeros(8, dtype=torch.int32))
    return gdn.KVCache(**dict(t, **changes))


def test_the_cache_object_checks_its_tensors():
    good = cpu_cache()
    with pytest.raises(AttributeError):
        good.k = good.v
    i32 = dict(dtype=torch.int32)
    for bad in (dict(k=torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)), dict(v=good.k[:, :4]),
                dict(table=torch.zeros(4, **i32)), dict(lengths=torch.zeros(5, **i32)),
                dict(refs=torch.zeros(9, **i32)), dict(k_scale=torch.zeros(1, 8, 2, 16))):
        with pytest.raises(ValueError):
            cpu_cache(**bad)
    with pytest.raises(TypeError):
        cpu_cache(k=good.k.float(), v=good.v.float())
    with pytest.raises(TypeError):
        cpu_cache(lengths=good.lengths.long())
    with pytest.raises(TypeError):
        gdn.kv_cache(1, 8, 2, 4, 3, dtype=torch.float16, device="cpu")
    for call in (lambda: gdn.cache_reserve(None, good.lengths), lambda: gdn.cache_free("x", good.refs),
                 lambda: gdn.attention_decode_step(good.k, good.k)):
        with pytest.raises(TypeError):
            call()


def test_the_binding_refuses_before_the_library():
    """Wrong types, shapes, strides and devices raise; CPU tensors are named as such."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    q, k = bf(6, 4, 64), bf(6, 2, 64)
    cu = torch.tensor([0, 6], dtype=torch.int32)
    with pytest.raises(TypeError):
        gdn.attention_prefill(q.float(), k, k)
    for args in ((q, bf(6, 2, 32), k), (q, k, bf(5, 2, 64)), (q, k[None], k[None]), (q[0], k, k),
                 (q, k, k, None, cu), (q, bf(7, 2, 64), bf(7, 2, 64), cu), (q, k, k, cu, cu[:1]),
                 (q, k, k, cu.reshape(1, 2)), (q.expand(6, 4, 64)[:, :, ::2], k, k),
                 (q.transpose(0, 1), k, k), (q[:1].expand(6, 4, 64), k, k),
                 (bf(2, 6, 4, 64), bf(3, 6, 2, 64), bf(3, 6, 2, 64)),
                 (bf(2, 6, 4, 64), bf(2, 6, 2, 64), bf(2, 6, 2, 64), cu)):
        with pytest.raises(ValueError):
            gdn.attention_prefill(*args)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.attention_prefill(q, k, k, cu)
    out, lse = bf(6, 4, 64), torch.zeros(6, 4)
    with pytest.raises(ValueError):
        gdn.attention_prefill_backward(q, k, k, out[:5], lse, out)
    with pytest.raises(TypeError):
        gdn.attention_prefill_backward(q, k, k, out, lse.double(), out)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.attention_prefill_backward(q, k, k, out, lse, out)
    with pytest.raises(ValueError):
        gdn.attention_prefill_backward_workspace_size(1, 6, 4, 3, 64)
    with pytest.raises(ValueError):
        gdn.attention_decode_step_workspace_size(1, 4, 3, 64)
    c = cpu_cache()
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    for call in (lambda: gdn.cache_reserve(c, i(1, 1)), lambda: gdn.cache_append(c, k, k, i(0, 0, 0, 0)),
                 lambda: gdn.cache_append(c, bf(4, 3, 64), bf(4, 3, 64), i(0, 0, 0, 0)),
                 lambda: gdn.cache_append(c, bf(4, 2, 64), bf(4, 2, 64), i(0, 0, 0)),
                 lambda: gdn.cache_append(c, k, k, i(0, 0, 0, 0), i(0, 1, 2)),
                 lambda: gdn.cache_free(c, i(0).reshape(1, 1)), lambda: gdn.cache_fork(c, i(0), i(1, 2)),
                 lambda: gdn.attention_decode_step(bf(3, 4, 64), c),
                 lambda: gdn.attention_decode_step(bf(4, 4, 32), c)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gdn.cache_reserve(c, i(1, 1, 1, 1).long()), lambda: gdn.cache_free(c, c.refs.float())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: gdn.cache_reserve(c, i(1, 1, 1, 1)), lambda: gdn.cache_free(c, i(0)),
                 lambda: gdn.attention_decode_step(bf(4, 4, 64), c)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
