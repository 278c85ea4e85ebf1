"""One decoder layer around the Gated DeltaNet mixer, built from the library's
calls: prompts and single tokens with 8-bit projections, and the training step
of its feed-forward half.

    python examples/decoder_layer.py

prefills a batch of prompts, decodes a few tokens from the states that the
prefill left, checks the decoded outputs against a prefill of the longer
prompts, and takes the gradients of the feed-forward half.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hybrid_linear_attention_deltanet_gb300 as gdn  # noqa: E402

EPS = 1e-5


class DecoderLayer:
    """dim -> mixer (heads x 256) -> dim -> gated feed-forward (hidden) -> dim.

    Projections are e4m3 with 128 x 128 block scales; the feed-forward's gate
    and up projections stay bf16.  The residual stream and the layer's output
    travel side by side, so that each norm adds the one to the other."""

    def __init__(self, dim=512, heads=2, hidden=1024, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.dim, self.heads, self.hidden, self.dv = dim, heads, hidden, 256
        self.channels = heads * 768                       # q | k | v
        eight = lambda n, k: gdn.quantize_fp8((rand(n, k) * k ** -0.5).bfloat16(),  # noqa: E731
                                              block_rows=128)
        self.w_qkv = eight(self.channels, dim)
        self.w_ab = eight(2 * heads, dim)                 # decay and write-strength inputs
        self.w_g = eight(heads * self.dv, dim)            # read-out gate
        self.w_o = eight(dim, heads * self.dv)
        self.w_down = eight(dim, hidden)
        self.w_gate = (rand(hidden, dim) * dim ** -0.5).bfloat16()
        self.w_up = (rand(hidden, dim) * dim ** -0.5).bfloat16()
        self.norm1, self.norm2 = 1 + 0.1 * rand(dim), 1 + 0.1 * rand(dim)
        self.conv_w = rand(self.channels, 4) * 0.5
        self.A_log, self.dt_bias = rand(heads) * 0.1, rand(heads) * 0.1
        self.norm_o = 1 + 0.1 * rand(self.dv)

    def _project(self, x, residual):
        """The mixer's inputs from the layer's: norm into 8 bits, three products."""
        q, s, res = gdn.residual_norm_fp8(x, self.norm1, residual, EPS)
        qkv = gdn.linear_fp8(q, s, *self.w_qkv)
        ab = gdn.linear_fp8(q, s, *self.w_ab, out_dtype=torch.float32)
        a, b = (t.contiguous() for t in ab.split(self.heads, -1))
        gate = gdn.linear_fp8(q, s, *self.w_g).unflatten(-1, (self.heads, self.dv))
        return qkv, a, b, gate, res

    def _finish(self, y, res):
        """The mixer's output back to the residual stream, then the feed-forward."""
        o = gdn.linear_fp8(*gdn.quantize_fp8(y.flatten(-2)), *self.w_o)
        z, res = gdn.residual_norm(o, self.norm2, res, EPS)
        h = gdn.gated_ffn(z, self.w_gate, self.w_up)
        return gdn.linear_fp8(*gdn.quantize_fp8(h), *self.w_down), res

    def prefill(self, x, residual=None):
        """x [B, T, dim] bf16 -> (out, residual stream, (conv state, S)) for whole prompts."""
        qkv, a, b, gate, res = self._project(x, residual)
        conv = torch.empty(x.shape[0], 3, self.channels, dtype=x.dtype, device=x.device)
        y, S = gdn.prefill_layer(qkv, self.conv_w, a, b, self.A_log, self.dt_bias, gate,
                                 self.norm_o, self.heads, conv_state_out=conv, eps=EPS)
        out, res = self._finish(y, res)
        return out, res, (conv, S)

    def decode(self, x, state, residual=None):
        """One token a sequence, x [B, dim]; the state is updated in place."""
        qkv, a, b, gate, res = self._project(x, residual)
        conv, S = state
        y = gdn.decode_layer_step(qkv, self.conv_w, a, b, self.A_log, self.dt_bias, conv, S, gate,
                                  self.norm_o, EPS)
        return self._finish(y, res)

    def train_feed_forward(self, o, residual, dh, dres=None):
        """Forward and backward of the feed-forward half up to its hidden
        activations h: o is the mixer's output, residual the stream it joins, dh
        the gradient of h and dres that of the stream from the layers above.
        Returns (h, gradients of o (and residual), norm2, w_gate, w_up)."""
        z, s = gdn.residual_norm(o, self.norm2, residual, EPS)
        h = gdn.gated_ffn(z, self.w_gate, self.w_up)
        f = gdn.gated_ffn_backward(z, self.w_gate, self.w_up, dh)
        n = gdn.residual_norm_backward(f["dx"], s, self.norm2, dres, EPS)
        return h, n["dx"], n["dw"], f["dw_gate"], f["dw_up"]


def main():
    layer = DecoderLayer()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 70, layer.dim, generator=g, device="cuda").bfloat16()
    whole, stream, _ = layer.prefill(x)
    _, _, state = layer.prefill(x[:, :64].contiguous())
    for t in range(64, 70):
        out, res = layer.decode(x[:, t].contiguous(), state)
        off = (out.float() - whole[:, t].float()).norm() / whole[:, t].float().norm()
        print(f"token {t}: decoded output against the prefill's, relative {off:.1e}")
    dh = torch.randn(2, 70, layer.hidden, generator=g, device="cuda").bfloat16()
    h, d_o, d_norm, d_gate, d_up = layer.train_feed_forward(whole, stream, dh, stream)
    print("gradient norms: o %.3g, norm %.3g, gate %.3g, up %.3g" % tuple(
        float(t.float().norm()) for t in (d_o, d_norm, d_gate, d_up)))
    if gdn.device_status() != 0:
        raise RuntimeError("the device reported an error")


if __name__ == "__main__":
    main()
