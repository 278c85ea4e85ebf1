"""What the binding hands to the C calls as plain addresses and integers is checked first: a
workspace's device."""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn


def test_a_workspace_of_another_device_is_refused():
    host = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        gdn._ws_args(host, 0)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        gdn._ws(host, 1)


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
