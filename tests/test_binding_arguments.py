"""What the binding hands to the C calls as plain addresses and integers is checked first: a
workspace's device, and integers that do not fit in 32 bits."""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn


def test_a_workspace_of_another_device_is_refused():
    host = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        gdn._ws_args(host, 0)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        gdn._ws(host, 1)


@pytest.mark.parametrize("far", [2 ** 32, 2 ** 32 + 1, 2 ** 31, -2 ** 32])
def test_integers_beyond_32_bits_are_refused(far):
    """They would be cut: 2^32 to layer 0, 2^32 + 1 sequences to one."""
    zeros = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)  # noqa: E731
    k, q = zeros(1, 8, 2, 16, 64, t=torch.bfloat16), zeros(4, 4, 64, t=torch.bfloat16)
    cache = gdn.KVCache(k, k.clone(), zeros(4, 3), zeros(4), zeros(8))
    for call in (lambda: gdn.attention_decode_step(q, cache, far),
                 lambda: gdn.cache_append(cache, q[:, :2].contiguous(), q[:, :2].contiguous(), zeros(4),
                                          layer=far),
                 lambda: gdn.cache_gather(cache, zeros(5), 1, layer=far),
                 lambda: gdn.attention_prefill_backward_workspace_size(far, 1, 1, 1, 64),
                 lambda: gdn.attention_prefill_backward_workspace_size(1, 1, 1, 1, far),
                 lambda: gdn.attention_decode_step_workspace_size(far, 1, 1, 64)):
        with pytest.raises(ValueError, match="out of range"):
            call()


def test_a_table_wider_than_32_bits_is_refused():
    meta = lambda *s, t=torch.int32: torch.empty(*s, dtype=t, device="meta")  # noqa: E731
    k = meta(1, 8, 2, 16, 64, t=torch.bfloat16)
    with pytest.raises(ValueError, match="max_pages .* out of range"):
        gdn.KVCache(k, k, meta(1, 2 ** 32 + 1), meta(1), meta(8))


@pytest.mark.gpu
def test_every_call_refuses_a_workspace_on_the_host(gdn_lib):
    before = gdn.kernel_launches()
    new = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    host = torch.zeros(1 << 24, dtype=torch.uint8)
    q, a = new(1, 64, 1, 256), new(1, 64, 1, t=torch.float32)
    x, w = new(128, 128), new(128, 128)
    h, lse = new(16, 2, 64), new(16, 2, t=torch.float32)
    cache = gdn.kv_cache(1, 4, 2, 16, 1, 16, 64)
    for call in (lambda: gdn.prefill(q, q, q, a, a, workspace=host),
                 lambda: gdn.prefill_scan(q, q, q, a, a, segments=1, workspace=host),
                 lambda: gdn.prefill_backward(q, q, q, a, a, q, workspace=host),
                 lambda: gdn.residual_norm_backward(x, x, new(128, t=torch.float32), workspace=host),
                 lambda: gdn.gated_ffn_backward(x, w, w, x, workspace=host),
                 lambda: gdn.attention_prefill_backward(h, h, h, h, lse, h, workspace=host),
                 lambda: gdn.attention_decode_step(h, cache, workspace=host)):
        with pytest.raises(ValueError, match="workspace is on cpu"):
            call()
    assert gdn.kernel_launches() == before
