"""An attention layer as a hybrid keeps among its Gated DeltaNet layers, built from the library's
calls: prompts and single tokens with 8-bit projections and a paged cache, forked answers, and the
gradients of its core.

    python examples/attention_layer.py

prefills a batch of prompts of different lengths into the cache, decodes a few tokens, forks one
prompt into three answers, checks the decoded outputs against a prefill of the longer prompts, and
takes the gradients of the attention.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hybrid_linear_attention_deltanet_gb300 as gdn  # noqa: E402

EPS = 1e-5


class AttentionLayer:
    """dim -> q | k | v (grouped heads of 128) -> attention -> dim, behind a residual norm.

    The projections are e4m3 with 128 x 128 block scales.  Position encodings are the
    caller's: q and k reach the attention as the projection leaves them."""

    def __init__(self, dim=512, heads=4, kv_heads=2, d=128, layer=0, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.heads, self.kv, self.d, self.layer = heads, kv_heads, d, layer
        eight = lambda n, k: gdn.quantize_fp8((rand(n, k) * k ** -0.5).bfloat16(),  # noqa: E731
                                              block_rows=128)
        self.w_qkv = eight((heads + 2 * kv_heads) * d, dim)
        self.w_o = eight(dim, heads * d)
        self.norm = 1 + 0.1 * rand(dim)

    def project(self, x, residual):
        """x [tokens, dim] -> q, k, v as slices of the packed projection, the residual stream."""
        z, s, res = gdn.residual_norm_fp8(x, self.norm, residual, EPS)
        qkv = gdn.linear_fp8(z, s, *self.w_qkv).unflatten(-1, (-1, self.d))
        return (*qkv.split((self.heads, self.kv, self.kv), -2), res)

    def output(self, o):
        return gdn.linear_fp8(*gdn.quantize_fp8(o.flatten(-2)), *self.w_o)

    def prefill(self, x, cu_seqlens, cache, start, residual=None):
        """Whole prompts, packed: x [tokens, dim], row r of the cache taking the tokens
        cu_seqlens[r] .. cu_seqlens[r + 1] from position start[r] = 0 on."""
        q, k, v, res = self.project(x, residual)
        gdn.cache_append(cache, k, v, start, cu_seqlens, self.layer)
        out, _ = gdn.attention_prefill(q, k, v, cu_seqlens)
        return self.output(out), res

    def prefill_on(self, x, cu_seqlens, cache, start, cu_all, tokens, residual=None):
        """Prompts that go on behind what their rows hold: x are the new tokens, cu_all and
        tokens the rows' lengths with them.  A row whose reservation failed (start -1) attends to
        zeros in the place of its new tokens; gdn.device_status() tells the caller."""
        q, k, v, res = self.project(x, residual)
        gdn.cache_append(cache, k, v, start, cu_seqlens, self.layer)
        k, v = gdn.cache_gather(cache, cu_all, tokens, self.layer)
        out, _ = gdn.attention_prefill(q, k, v, cu_seqlens, cu_all)
        return self.output(out), res

    def decode(self, x, cache, start, residual=None):
        """One token a row, x [rows, dim]; its place was reserved for all layers at once."""
        q, k, v, res = self.project(x, residual)
        gdn.cache_append(cache, k, v, start, layer=self.layer)
        return self.output(gdn.attention_decode_step(q.contiguous(), cache, self.layer)), res

    def train_core(self, x, cu_seqlens, dout, residual=None):
        """Forward and backward of the attention between its projections: dout is the gradient of
        its output [tokens, heads, d].  Returns (out, dict dq, dk, dv)."""
        q, k, v, _ = self.project(x, residual)
        out, lse = gdn.attention_prefill(q, k, v, cu_seqlens)
        return out, gdn.attention_prefill_backward(q, k, v, out, lse, dout, cu_seqlens)


def main():
    dim, rows, lens, more = 512, 8, [70, 33, 129], 5
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = [torch.randn(n + more, dim, generator=g, device="cuda").bfloat16() for n in lens]
    n = len(lens)

    for dtype in (torch.bfloat16, torch.float8_e4m3fn):
        layer = AttentionLayer(dim)
        cache = gdn.kv_cache(1, 32, layer.kv, rows, 4, page=64, d=layer.d, dtype=dtype)
        counts = lens + [0] * (rows - n)
        cu = ints([sum(counts[:i]) for i in range(rows + 1)])
        start = gdn.cache_reserve(cache, ints(counts))
        layer.prefill(torch.cat([t[:m] for t, m in zip(x, lens)]), cu, cache, start)
        # the first prompt goes on in three rows besides its own
        gdn.cache_fork(cache, ints([0, 0, 0]), ints([n, n + 1, n + 2]))
        one = ints([1] * (n + 3) + [0] * (rows - n - 3))
        for t in range(more):
            now = [x[i][lens[i] + t] for i in range(n)] + [x[0][lens[0] + t]] * 3
            now = torch.stack(now + [torch.zeros_like(x[0][0])] * (rows - n - 3))
            out, _ = layer.decode(now, cache, gdn.cache_reserve(cache, one))
        whole, _ = layer.prefill(torch.cat(x), ints([0] + [sum(m + more for m in lens[:i + 1])
                                                           for i in range(n)]),
                                 gdn.kv_cache(1, 32, layer.kv, n, 4, d=layer.d),
                                 ints([-1] * n))     # (nothing is kept of this one)
        last = [sum(m + more for m in lens[:i + 1]) - 1 for i in range(n)]
        want = whole[last + [last[0]] * 3].float()
        off = (out[:n + 3].float() - want).norm() / want.norm()
        # the same tokens as a next turn of whole prompts
        again = gdn.kv_cache(1, 32, layer.kv, n, 4, page=64, d=layer.d, dtype=dtype)
        layer.prefill(torch.cat([t[:m] for t, m in zip(x, lens)]), cu[:n + 1].contiguous(), again,
                      gdn.cache_reserve(again, ints(lens)))
        turn, _ = layer.prefill_on(torch.cat([t[m:] for t, m in zip(x, lens)]),
                                   ints([more * i for i in range(n + 1)]), again,
                                   gdn.cache_reserve(again, ints([more] * n)),
                                   ints([sum(m + more for m in lens[:i]) for i in range(n + 1)]),
                                   sum(lens) + n * more)
        turn = turn[[more * (i + 1) - 1 for i in range(n)]].float()
        print(f"{str(dtype)[6:]} cache: a next turn's last tokens, relative "
              f"{(turn - want[:n]).norm() / want[:n].norm():.1e}")
        print(f"{str(dtype)[6:]} cache: decoded outputs against the prefill's, relative {off:.1e}; "
              f"{int((cache.refs > 0).sum())} pages held")

    dout = torch.randn(sum(lens), layer.heads, layer.d, generator=g, device="cuda").bfloat16()
    packed = torch.cat([t[:m] for t, m in zip(x, lens)])
    out, grads = layer.train_core(packed, ints([0, lens[0], lens[0] + lens[1], sum(lens)]), dout)
    print("gradient norms: q %.3g, k %.3g, v %.3g" % tuple(
        float(grads[n].float().norm()) for n in ("dq", "dk", "dv")))
    if gdn.device_status() != 0:
        raise RuntimeError("the device reported an error")


if __name__ == "__main__":
    main()
