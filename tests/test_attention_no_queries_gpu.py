"""Packed calls without a single query: malformed sequences are flagged and write nothing, as with
queries; well-formed ones give keys that no query sees zero gradients."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
BAD_SEQLENS = 6


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cq,ck,good", [
    ([0, 0, 0], [0, 5, 12], True), ([0, 0], [0, 12], True),
    ([0] * 3001, [0] * 1500 + [7] * 1500 + [12], True),
    ([0, 0, 0], [0, 5, 11], False), ([0, 0, 0], [0, 13, 12], False), ([0, 0, 0], [1, 5, 12], False),
    ([0, 1, 0], [0, 5, 12], False), ([0, 0, 1], [0, 5, 12], False), ([-1, 0, 0], [0, 5, 12], False),
    ([0] * 3001, [0] * 1500 + [-7] + [12] * 1500, False)])
def test_packed_without_queries(gdn_lib, cq, ck, good, d):
    gdn = gdn_lib
    q, k = (torch.randn(n, h, d, device="cuda").to(BF16) for n, h in ((0, 4), (12, 2)))
    cq, ck = ints(cq), ints(ck)
    out, lse = gdn.attention_prefill(q, k, k, cq, ck)
    assert out.shape == q.shape and gdn.device_status() == (0 if good else BAD_SEQLENS)
    dk, dv = torch.full_like(k, 7), torch.full_like(k, 7)
    gdn._call("gdn_attention_prefill_backward", k.get_device(), None, None, k.data_ptr(), k.data_ptr(),
              None, None, None, cq.data_ptr(), ck.data_ptr(), 0.1, None, dk.data_ptr(), dv.data_ptr(),
              len(cq) - 1, 0, 12, 4, 2, d, 4 * d, 2 * d, 2 * d)
    assert gdn.device_status() == (0 if good else BAD_SEQLENS)
    for t in (dk, dv):
        assert (t == (0 if good else 7)).all()
    g = gdn.attention_prefill_backward(q, k, k, out, lse, out, cq, ck)
    assert g["dq"].shape == q.shape and gdn.device_status() == (0 if good else BAD_SEQLENS)
    if good:
        assert (g["dk"] == 0).all() and (g["dv"] == 0).all()


def test_neither_queries_nor_keys(gdn_lib):
    gdn = gdn_lib
    q, k = (torch.zeros(0, h, 64, device="cuda", dtype=BF16) for h in (4, 2))
    for cu, status in (([0, 0, 0], 0), ([0, 3, 0], BAD_SEQLENS)):
        out, lse = gdn.attention_prefill(q, k, k, ints(cu))
        assert gdn.device_status() == status
        gdn.attention_prefill_backward(q, k, k, out, lse, out, ints(cu))
        assert gdn.device_status() == status
