"""Sizes next to 2^31: what the layer operators' 32-bit tile coordinates do not
hold is refused as unsupported on the host, before any launch.  Fake
addresses, so these run only where no CUDA device is visible."""
import ctypes

import pytest

import hybrid_linear_attention_deltanet_gb300 as gdn  # noqa: F401
from test_abi import fake_addresses, lib  # noqa: F401  (fixture)

P = ctypes.c_void_p
SIZE_MAX = ctypes.c_size_t(-1).value
BF16 = 1
# far enough apart for every size here
A, B, C, D, E, F, G = (P((i + 1) << 52) for i in range(7))
UNSUPPORTED = 2
TOP = 0x7ffffff8        # the largest multiple of 8 that an int32 holds


@fake_addresses
@pytest.mark.parametrize("hidden", [0x3fffff81, 0x40000001, 0x7fffff00, 0x7fffffff])
def test_feed_forward_hidden(lib, hidden):  # noqa: F811
    # a tile has two columns of the product for each feature
    assert lib.gdn_gated_ffn(A, B, C, 0, D, 16, 8, hidden, BF16, None) == UNSUPPORTED
    assert lib.gdn_gated_ffn_backward(A, B, C, D, 0, E, F, G, 16, 8, hidden, BF16,
                                      None) == UNSUPPORTED
    assert lib.gdn_gated_ffn_backward_workspace_size(16, 8, hidden, BF16) == SIZE_MAX


@fake_addresses
@pytest.mark.parametrize("dim", [0x7fffff08, TOP])
def test_inner_axes(lib, dim):  # noqa: F811
    assert lib.gdn_gated_ffn(A, B, C, 0, D, 16, dim, 8, BF16, None) == UNSUPPORTED
    assert lib.gdn_gated_ffn_backward(A, B, C, D, 0, E, F, G, 16, dim, 8, BF16,
                                      None) == UNSUPPORTED
    assert lib.gdn_gated_ffn_backward_workspace_size(16, dim, 8, BF16) == SIZE_MAX
    assert lib.gdn_quantize_fp8(A, B, C, 16, dim, 1, BF16, None) == UNSUPPORTED
    assert lib.gdn_quantize_fp8(A, B, C, 16, dim, 128, BF16, None) == UNSUPPORTED
    k = dim & ~15
    assert lib.gdn_linear_fp8(A, B, C, D, E, 16, max(k, 0x7fffff10), 8, BF16, None) == UNSUPPORTED


@fake_addresses
def test_sizes_below_are_not_refused_for_their_size(lib):  # noqa: F811
    """They get as far as the device (which is missing here)."""
    CUDA = 4
    assert lib.gdn_gated_ffn(A, B, C, 0, D, 16, 8, 0x3fffff80, BF16, None) == CUDA
    assert lib.gdn_linear_fp8(A, B, C, D, E, 16, 0x7fffff00, 8, BF16, None) == CUDA
