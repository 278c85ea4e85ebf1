"""What is measured of the operators around the Gated DeltaNet mixer of a decoder layer, and their
plain forms: the residual addition with its root-mean-square norm (8-bit output for serving, its
gradient for training), the block-scaled 8-bit matrix product, and the gated feed-forward
projections with their gradients.

Formulas (rows t are tokens):
  norm      s = round(x + r);  y = s / sqrt(mean_j s_j^2 + eps) * w
  8 bits    per row and block of 128 columns: m = max(|y|, 2^-100), scale = m / 448,
            q = e4m3(y * (448 / m)), a value being q * scale
  gradient  n = s / rms;  g = dy * w;  dx = (g - n mean_j(g n)) / rms + ds;  dw = sum_t dy n
  product   out[t, n] = sum_k (xq sx)[t, k] (wq sw)[n, k], scales per 1 x 128 of x, 128 x 128 of w
  gated     G = x Wg^T, U = x Wu^T, h = act(G) U;
            dU = dh act(G), dG = dh U act'(G), dx = dG Wg + dU Wu, dWg = dG^T x, dWu = dU^T x
"""
import torch

own = False

EPS = 1e-5
BLOCK = 128
E4M3 = torch.float8_e4m3fn
BF16 = torch.bfloat16


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence's next token enters a layer: the serving step's norm, where latency counts
        dict(name="norm_fp8_1", op="norm_fp8", tokens=1, dim=2048, residual=True),
        # the training-length batch (4 x 8192 tokens) on its way into the 8-bit projections
        dict(name="norm_fp8_32k", op="norm_fp8", tokens=32768, dim=2048, residual=True),
        # a training step's norm gradient, an odd number of tokens and a wider residual stream
        dict(name="norm_backward_8191", op="norm_backward", tokens=8191, dim=4096, residual=True),
        # the packed q|k|v projection (6 heads: 4608 channels) of one sequence's next token
        dict(name="linear_1", op="linear_fp8", tokens=1, k=2048, n=4608, raw=False),
        # the same for 256 sequences decoding together
        dict(name="linear_256", op="linear_fp8", tokens=256, k=2048, n=4608, raw=False),
        # the same at prefill: 4 x 8192 tokens
        dict(name="linear_32k", op="linear_fp8", tokens=32768, k=2048, n=4608, raw=False),
        # the mixer's output (bf16, quantised in the call) back to the model: a ragged prompt,
        # sizes that are no multiple of a block or a tile
        dict(name="linear_ragged", op="linear_fp8", tokens=3001, k=1552, n=2005, raw=True),
        # feed-forward of one sequence's next token: reads the two weights
        dict(name="ffn_1", op="ffn", tokens=1, dim=2048, hidden=6144, act="silu"),
        # feed-forward of 256 sequences decoding together
        dict(name="ffn_256", op="ffn", tokens=256, dim=2048, hidden=6144, act="silu"),
        # feed-forward at prefill and in a training step's forward pass
        dict(name="ffn_32k", op="ffn", tokens=32768, dim=2048, hidden=6144, act="silu"),
        # its gradients for one 8K sequence
        dict(name="ffn_backward_8k", op="ffn_backward", tokens=8192, dim=2048, hidden=6144,
             act="silu"),
        # its gradients at a short ragged batch, odd sizes, the logistic gate
        dict(name="ffn_backward_ragged", op="ffn_backward", tokens=1111, dim=1032, hidden=2731,
             act="sigmoid"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(lo * (hi / lo) ** rng.random()))
    return n if n != 3072 else n + 1


def draw(rng):
    op = rng.choice(["norm_fp8", "norm_backward", "linear_fp8", "linear_fp8", "ffn", "ffn_backward"])
    if op in ("norm_fp8", "norm_backward"):
        dim = 16 * _log_int(rng, 32, 320)
        most = 32768 * 2048 // dim if op == "norm_fp8" else 8191 * 4096 // dim
        return dict(op=op, tokens=_log_int(rng, 1, most), dim=dim + (16 if dim == 3072 else 0),
                    residual=rng.random() < 0.75)
    if op == "linear_fp8":
        k, n = 16 * _log_int(rng, 16, 320), _log_int(rng, 12, 8192)
        k += 16 if k == 3072 else 0
        most = max(1, min(32768, 32768 * 2048 * 4608 // (k * n), 32768 * 4608 // n))
        return dict(op=op, tokens=_log_int(rng, 1, most), k=k, n=n, raw=rng.random() < 0.5)
    dim, hidden = 8 * _log_int(rng, 32, 512), _log_int(rng, 256, 8192)
    dim += 8 if dim == 3072 else 0
    most = 32768 if op == "ffn" else 8192
    most = max(1, min(most, most * 2048 * 6144 // (dim * hidden), most * 6144 // hidden))
    return dict(op=op, tokens=_log_int(rng, 1, most), dim=dim, hidden=hidden,
                act=rng.choice(["silu", "silu", "sigmoid"]))


# ----------------------------------------------------------------------------------- inputs
def _quantise_plain(y, block_rows):
    """y [R, C] fp32 -> (e4m3 codes [R, C], fp32 scales [ceil(R / block_rows), ceil(C / 128)])."""
    rows, cols = y.shape
    nr, nc = -(-rows // block_rows), -(-cols // BLOCK)
    p = torch.zeros(nr * block_rows, nc * BLOCK, dtype=torch.float32, device=y.device)
    p[:rows, :cols] = y
    b = p.view(nr, block_rows, nc, BLOCK)
    m = b.abs().amax(dim=(1, 3)).clamp_min(2.0 ** -100)
    q = (b * (448.0 / m)[:, None, :, None]).view_as(p)[:rows, :cols].to(E4M3)
    return q.contiguous(), m / 448.0


def _activations(g, tokens, dim):
    """Unit-variance activations with a few louder channels, as a residual stream has them."""
    x = torch.randn(tokens, dim, generator=g, device="cuda")
    loud = torch.randint(0, dim, (max(1, dim // 128),), generator=g, device="cuda")
    x[:, loud] *= 8.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op, T = case["op"], case["tokens"]
    s = dict(case=case)
    if op in ("norm_fp8", "norm_backward"):
        D = case["dim"]
        s["w"] = 1.0 + 0.1 * rand(D)
        if op == "norm_fp8":
            s["x"] = rand(T, D).to(BF16)
            s["residual"] = _activations(g, T, D).to(BF16) if case["residual"] else None
        else:
            s["s"] = _activations(g, T, D).to(BF16)
            s["dy"] = (0.1 * rand(T, D)).to(BF16)
            s["ds"] = (0.1 * rand(T, D)).to(BF16) if case["residual"] else None
    elif op == "linear_fp8":
        K, N = case["k"], case["n"]
        x = _activations(g, T, K).to(BF16)
        if case["raw"]:
            s["x"] = x
        else:
            s["xq"], s["sx"] = _quantise_plain(x.float(), 1)
        s["wq"], s["sw"] = _quantise_plain(rand(N, K) * K ** -0.5, BLOCK)
    else:
        D, F = case["dim"], case["hidden"]
        s["x"] = rand(T, D).to(BF16)
        s["wg"] = (rand(F, D) * D ** -0.5).to(BF16)
        s["wu"] = (rand(F, D) * D ** -0.5).to(BF16)
        if op == "ffn_backward":
            s["dh"] = (0.1 * rand(T, F)).to(BF16)
    return s


# -------------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state, state["case"]["op"])


def _run_own(s, op):
    import hybrid_linear_attention_deltanet_gb300 as gdn
    if op == "norm_fp8":
        q, scale, sums = gdn.residual_norm_fp8(s["x"], s["w"], s["residual"], EPS)
        return dict(q=q, scale=scale, sum=sums)
    if op == "norm_backward":
        r = gdn.residual_norm_backward(s["dy"], s["s"], s["w"], s["ds"], EPS)
        return dict(dx=r["dx"], dw=r["dw"])
    if op == "linear_fp8":
        xq, sx = gdn.quantize_fp8(s["x"]) if s["case"]["raw"] else (s["xq"], s["sx"])
        return dict(out=gdn.linear_fp8(xq, sx, s["wq"], s["sw"]))
    if op == "ffn":
        return dict(h=gdn.gated_ffn(s["x"], s["wg"], s["wu"], s["case"]["act"]))
    r = gdn.gated_ffn_backward(s["x"], s["wg"], s["wu"], s["dh"], s["case"]["act"])
    return dict(dx=r["dx"], dwg=r["dw_gate"], dwu=r["dw_up"])


def _spread(scale, rows, cols, block_rows):
    """Block scales [R', C'] as one factor per element [rows, cols]."""
    if block_rows > 1:
        scale = scale.repeat_interleave(block_rows, 0)[:rows]
    return scale.repeat_interleave(BLOCK, 1)[:, :cols]


def _gate(G, act):
    sg = 1.0 / (1.0 + torch.exp(-G))
    if act == "silu":
        return G * sg, sg * (1.0 + G * (1.0 - sg))
    return sg, sg * (1.0 - sg)


def _run_plain(s, op):
    if op == "norm_fp8":
        x = s["x"]
        sums = x if s["residual"] is None else (x.float() + s["residual"].float()).to(BF16)
        f = sums.float()
        y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["w"]
        q, scale = _quantise_plain(y, 1)
        return dict(q=q, scale=scale, sum=sums)
    if op == "norm_backward":
        f, dy = s["s"].float(), s["dy"].float()
        inv = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        n, gw = f * inv, dy * s["w"]
        dx = (gw - n * (gw * n).mean(-1, keepdim=True)) * inv
        if s["ds"] is not None:
            dx = dx + s["ds"].float()
        return dict(dx=dx.to(BF16), dw=(dy * n).sum(0))
    if op == "linear_fp8":
        xq, sx = _quantise_plain(s["x"].float(), 1) if s["case"]["raw"] else (s["xq"], s["sx"])
        (T, K), N = xq.shape, s["wq"].shape[0]
        x = xq.float() * _spread(sx, T, K, 1)
        w = s["wq"].float() * _spread(s["sw"], N, K, BLOCK)
        return dict(out=(x @ w.t()).to(BF16))
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    G, U = x @ wg.t(), x @ wu.t()
    a, da = _gate(G, s["case"]["act"])
    if op == "ffn":
        return dict(h=(a * U).to(BF16))
    dh = s["dh"].float()
    dU, dG = dh * a, dh * U * da
    return dict(dx=(dG @ wg + dU @ wu).to(BF16), dwg=(dG.t() @ x).to(BF16),
                dwu=(dU.t() @ x).to(BF16))


# ---------------------------------------------------------------- from the definition, 64 bits
def _e4m3_64(v):
    """Nearest e4m3 value of |v| <= 448 in 64 bits, ties to even: 3 fraction bits, exponents
    from -6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _blocks_64(y, codes):
    """(codes, scales) of 1 x 128 blocks, column block by column block."""
    q, scale = torch.empty_like(y), []
    for c in range(0, y.shape[1], BLOCK):
        b = y[:, c:c + BLOCK]
        m = torch.clamp(b.abs().max(dim=1, keepdim=True).values, min=2.0 ** -100)
        q[:, c:c + BLOCK] = codes(b / m * 448.0)
        scale.append(m / 448.0)
    return q, torch.cat(scale, 1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "norm_fp8":
        t = d["x"] + d["residual"] if "residual" in d else d["x"]
        t = t.to(BF16).double()
        rms = torch.sqrt(torch.sum(t ** 2, -1, keepdim=True) / t.shape[1] + EPS)
        q, scale = _blocks_64(t / rms * d["w"], _e4m3_64)
        return dict(q=q, scale=scale, sum=t)
    if op == "norm_backward":
        rms = torch.sqrt(torch.sum(d["s"] ** 2, -1, keepdim=True) / d["s"].shape[1] + EPS)
        gw = d["dy"] * d["w"]
        along = torch.sum(gw * d["s"], -1, keepdim=True) / (d["s"].shape[1] * rms ** 2)
        dx = (gw - d["s"] * along) / rms
        return dict(dx=dx + d["ds"] if "ds" in d else dx, dw=torch.sum(d["dy"] * d["s"] / rms, 0))
    if op == "linear_fp8":
        if case["raw"]:
            # the codes are part of the operator: those of the call's own rule
            xq, sx = _blocks_64(d["x"], _e4m3_64)
        else:
            xq, sx = d["xq"], d["sx"]
        out = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
        for i in range(sx.shape[1]):
            cols = slice(i * BLOCK, (i + 1) * BLOCK)
            rows = torch.arange(case["n"], device="cuda") // BLOCK
            out += (xq[:, cols] * sx[:, i:i + 1]) @ (d["wq"][:, cols] * d["sw"][rows, i:i + 1]).T
        return dict(out=out)
    G, U = torch.einsum("td,fd->tf", d["x"], d["wg"]), torch.einsum("td,fd->tf", d["x"], d["wu"])
    sg = torch.sigmoid(G)
    a = G * sg if case["act"] == "silu" else sg
    if op == "ffn":
        return dict(h=a * U)
    da = sg + G * sg * torch.sigmoid(-G) if case["act"] == "silu" else sg * torch.sigmoid(-G)
    dU, dG = d["dh"] * a, d["dh"] * U * da
    return dict(dx=torch.einsum("tf,fd->td", dG, d["wg"]) + torch.einsum("tf,fd->td", dU, d["wu"]),
                dwg=torch.einsum("tf,td->fd", dG, d["x"]), dwu=torch.einsum("tf,td->fd", dU, d["x"]))


# ------------------------------------------------------------------------------------- work
def work(case):
    op, T = case["op"], case["tokens"]
    if op == "norm_fp8":
        D, blocks = case["dim"], -(-case["dim"] // BLOCK)
        read = T * D * (4 if case["residual"] else 2) + 4 * D
        return dict(bytes=read + T * D * 3 + T * blocks * 4, flops=8 * T * D)
    if op == "norm_backward":
        D = case["dim"]
        return dict(bytes=T * D * (8 if case["residual"] else 6) + 8 * D, flops=14 * T * D)
    if op == "linear_fp8":
        K, N = case["k"], case["n"]
        blocks = -(-K // BLOCK)
        x = 2 * T * K if case["raw"] else T * (K + 4 * blocks)
        return dict(bytes=x + N * K + -(-N // BLOCK) * blocks * 4 + 2 * T * N, flops=2 * T * N * K)
    D, F = case["dim"], case["hidden"]
    if op == "ffn":
        return dict(bytes=2 * (T * D + 2 * F * D + T * F), flops=4 * T * D * F)
    # G and U again from the inputs, then the three gradients
    return dict(bytes=2 * (T * D + 2 * F * D + T * F) + 2 * (T * D + 2 * F * D), flops=12 * T * D * F)
