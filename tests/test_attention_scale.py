"""Scales up to 2^127 are taken; beyond, their product with log2 e is no fp32 number, and the call
is refused instead of answering with NaN."""
import ctypes

import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn
from test_abi import fake_addresses, lib  # noqa: F401  (fixture)
from test_attention_abi import A, cache

TOO_MUCH = [1.8e38, 2.4e38, 2.9e38, 3.4e38]


@fake_addresses
@pytest.mark.parametrize("scale", TOO_MUCH)
def test_refused(lib, scale):  # noqa: F811
    def prefill(scale):
        return lib.gdn_attention_prefill(*A[:3], None, None, scale, A[3], A[4], 1, 0, 4, 8, 2, 64, 512,
                                         128, 128, None)
    assert prefill(2.0 ** 127) == 0 and prefill(scale) == 1
    assert lib.gdn_attention_prefill_backward(*A[:6], None, None, scale, *A[6:9], 1, 0, 0, 8, 2, 64, 512,
                                              128, 128, None) == 1
    assert lib.gdn_attention_decode_step(A[11], ctypes.byref(cache()), 0, 4, scale, A[12], None) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** -126])
def test_the_largest_and_smallest(gdn_lib, scale):
    """Scores of zero stay zero, so every result is the values' mean over what the row sees."""
    n, d = 40, 64
    q = torch.zeros(n, 2, d, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(n, 1, d, device="cuda").to(torch.bfloat16)
    v = torch.ones(n, 1, d, device="cuda", dtype=torch.bfloat16)
    out, lse = gdn.attention_prefill(q, k, v, scale=scale)
    assert (out == 1).all()
    count = torch.arange(1, n + 1, device="cuda").double().log()[:, None]
    assert ((lse.double() - count).abs() <= 2.0 ** -16 * (1 + count)).all()
    g = gdn.attention_prefill_backward(q, k, v, out, lse, torch.ones_like(q), scale=scale)
    assert (g["dq"] == 0).all()         # dP = D: d ones in both
    cache_ = gdn.kv_cache(1, 3, 1, 1, 3, 16, d)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    gdn.cache_append(cache_, k, v, gdn.cache_reserve(cache_, ints([n])), ints([0, n]))
    assert (gdn.attention_decode_step(q[:1], cache_, scale=scale) == 1).all()
    assert gdn.device_status() == 0
