"""fp32 results of the 8-bit product hold fp32's bits.

Tolerances, from the arithmetic.  A product of two e4m3 values has 8 bits and
is exact.  A K block's sum takes four tensor-core steps of 32 products, each
addition of whose sums to the fp32 accumulator is off by 2^-23 of the largest
partial sum at most: 5 x 2^-23 of S = sum |a b|, the products' alignment within
a step among them.  The factor of two scales, its product with the block's sum
and the addition to those of the blocks before are 2^-24 each, of at most S:
(blocks + 2) 2^-24 S in all.  In norm, errors of independent signs add to
sqrt(5 + blocks) 2^-23 of a sum of terms that are so too, below 2^-20 for 40
blocks and fewer.  Sums held in bf16's or fp16's bits (2^-9, 2^-12) are far
outside both.
"""
import pytest
import torch

import hybrid_linear_attention_deltanet_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def spread(scale, rows, cols, block_rows):
    s = scale.double()
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols]


# one token, clusters that split K, a cluster each, pairs of either width
@pytest.mark.parametrize("tokens,k,n", [(1, 2048, 4608), (17, 5120, 300), (64, 400, 257),
                                        (256, 2048, 512), (300, 4096, 129), (513, 2048, 4608),
                                        (3001, 1552, 2005)])
def test_fp32_results(tokens, k, n):
    g = torch.Generator(device=DEV).manual_seed(tokens + k + n)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, sx = gdn.quantize_fp8(rand(tokens, k))
    w, sw = gdn.quantize_fp8(rand(n, k) * k ** -0.5, block_rows=128)
    out = gdn.linear_fp8(x, sx, w, sw, F32).double()
    xd, wd = x.double() * spread(sx, tokens, k, 1), w.double() * spread(sw, n, k, 128)
    ref, S = xd @ wd.T, xd.abs() @ wd.abs().T
    blocks = -(-k // 128)
    over = (out - ref).abs() - (5 * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24) * S
    assert float(over.max()) <= 0
    assert float((out - ref).norm() / ref.norm()) <= 2.0 ** -20
