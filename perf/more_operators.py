"""What is measured of the attention layers that a hybrid keeps beside its Gated DeltaNet mixers, and
their plain forms: attention over whole prompts and its gradients, attention of one new token over
a paged cache, and the cache's pages (appending, forking, compacting).

Formulas (per sequence and query head; the kv head is the query head / group):
  prefill   s_ij = scale q_i . k_j for j <= i + len_k - len_q;  lse_i = log sum_j exp(s_ij);
            o_i = sum_j exp(s_ij - lse_i) v_j;  a row that sees no key: o = 0, lse = -inf
  gradient  P = exp(s - lse), D_i = do_i . o_i, dS = P (do_i . v_j - D_i);
            dq = scale dS k, dk = scale dS^T q, dv = P^T do (dk, dv summed over a group's heads)
  decode    the last row of the above, keys and values through the rows' page tables
  pages     a cache holds k and v [layers, pages, kv heads, page, d], a table of page numbers and
            a length for each row, and a reference count for each page (0: free).  Pages are
            taken in the order of their numbers, for the rows in the order given.
  8 bits    a cached key or value as e4m3 codes and a scale per token and head:
            m = max(|x|, 2^-100), scale = m / 448, code = e4m3(x * (448 / m))
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
BF16 = torch.bfloat16


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a chat's next turn: a few new tokens whose keys continue a stored context; latency counts
        dict(name="prefill_turn", op="prefill", q="17", k="1200", heads=16, kv=4, d=128),
        # prompts at the training length: 4 x 8192 tokens
        dict(name="prefill_4x8k", op="prefill", q="8192 8192 8192 8192", k="", heads=16, kv=4, d=128),
        # gradients of a short ragged batch: odd lengths and group, narrow heads
        dict(name="backward_ragged", op="backward", q="1000 24 333 1 2047", k="", heads=6, kv=2, d=64),
        # a training step's gradients: 2 x 8192 tokens
        dict(name="backward_2x8k", op="backward", q="8192 8192", k="", heads=16, kv=4, d=128),
        # one conversation about a long document, its next token: latency counts; 8-bit cache,
        # small pages, an odd group of heads
        dict(name="decode_1", op="decode", rows=1, most=32768, spread=0, heads=20, kv=4, d=128,
             page=32, bits=8),
        # 256 conversations of different lengths decoding together
        dict(name="decode_256", op="decode", rows=256, most=8192, spread=1, heads=16, kv=4, d=128,
             page=64, bits=16),
        # 256 rows' new keys and values into one layer's cache, every layer of every decoding step
        dict(name="append_token", op="append", rows=256, most=1024, prompt=False, kv=4, d=128,
             page=64, bits=16),
        # new prompts (4 rows of up to 8192 tokens) take the place of finished ones, 8-bit cache
        dict(name="append_prompts", op="append", rows=4, most=8192, prompt=True, kv=4, d=128,
             page=64, bits=8),
        # one prompt answered four times: three forks of a long row
        dict(name="fork_3", op="fork", sources=1, copies=3, most=8191, layers=7, kv=4, d=128,
             page=64, bits=16),
        # a beam step: 24 rows each continued by three others
        dict(name="fork_72", op="fork", sources=24, copies=3, most=4096, layers=7, kv=4, d=128,
             page=64, bits=16),
        # moving what lives of a fragmented pool to a smaller one, one layer, 8 bits
        dict(name="compact_small", op="compact", pages=512, live=0.5, layers=1, kv=4, d=128,
             page=64, bits=8),
        # the same for seven layers' pool
        dict(name="compact_7_layers", op="compact", pages=1536, live=0.6, layers=7, kv=4, d=128,
             page=64, bits=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _pairs(ql, kl):
    """Pairs (query, key) of the causal mask that ends at both last tokens."""
    first = max(0, ql - kl)                      # rows before this one see nothing
    n = ql - first
    return n * (kl - ql + first + 1) + n * (n - 1) // 2


def _lens(text):
    return [int(t) for t in text.split()]


def _seqs(case):
    ql = _lens(case["q"])
    return ql, _lens(case["k"]) if case["k"] else ql


_MOST_PAIRS = {"prefill": 4 * _pairs(8192, 8192) * 16 * 128, "backward": 2 * _pairs(8192, 8192) * 16 * 128}


def draw(rng):
    op = rng.choice(["prefill", "prefill", "backward", "backward", "decode", "decode", "append",
                     "fork", "compact"])
    d, kv, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
    page = rng.choice([16, 32, 64, 128])
    if op in ("prefill", "backward"):
        ql = [_log_int(rng, 1, 8192) for _ in range(rng.choice([1, 1, 2, 3, 5, 9]))]
        # (gradients of nothing but single tokens are zero)
        ql[0] = max(ql[0], 16) if op == "backward" else ql[0]
        if rng.random() < 0.5:
            kl = ql
        else:      # a stored context before the new tokens, now and then fewer keys than queries
            kl = [max(1, n + rng.choice([0, _log_int(rng, 1, 4096), -rng.randint(0, n // 2)]))
                  for n in ql]
        while sum(map(_pairs, ql, kl)) * kv * group * d > _MOST_PAIRS[op]:
            ql, kl = [(n + 1) // 2 for n in ql], [(n + 1) // 2 for n in kl]
        return dict(op=op, q=" ".join(map(str, ql)), k=" ".join(map(str, kl)) if kl != ql else "",
                    heads=kv * group, kv=kv, d=d)
    bits = rng.choice([8, 16])
    if op == "decode":
        most = _log_int(rng, 1, 32768)
        rows = _log_int(rng, 1, max(1, min(256, 2 ** 29 // (most * kv * d))))
        return dict(op=op, rows=rows, most=most, spread=rng.randint(0, 1), heads=kv * group, kv=kv,
                    d=d, page=page, bits=bits)
    if op == "append":
        prompt = rng.random() < 0.5
        rows = rng.randint(1, 12) if prompt else _log_int(rng, 1, 256)
        most = _log_int(rng, 1, 32768 // rows if prompt else 2 ** 18 // rows // (page // 16))
        return dict(op=op, rows=rows, most=most, prompt=prompt, kv=min(kv, 4), d=d, page=page, bits=bits)
    if op == "fork":
        return dict(op=op, sources=rng.randint(1, 24), copies=rng.randint(1, 3),
                    most=_log_int(rng, 1, 4096), layers=rng.randint(1, 7), kv=min(kv, 4), d=d,
                    page=min(page, 64), bits=bits)
    return dict(op=op, pages=_log_int(rng, 8, 1536), live=round(rng.uniform(0.1, 0.8), 2),
                layers=rng.randint(1, 7), kv=min(kv, 4), d=d, page=min(page, 64), bits=bits)


# ----------------------------------------------------------------------------------- inputs
def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _quantise(x):
    """x [.., d] -> (e4m3 codes, fp32 scales [..])."""
    m = x.float().abs().amax(-1).clamp_min(2.0 ** -100)
    return (x.float() * (448.0 / m)[..., None]).to(E4M3), m / 448.0


def _sizes(case):
    """Tokens in each row of the cache before the call, the case's own."""
    op, rng = case["op"], random.Random(1)
    if op == "decode":
        n = case["rows"]
        return [case["most"] if not case["spread"] or i == 0 else rng.randint(1, case["most"])
                for i in range(n)]
    if op == "append":
        # decoding rows; or rows that finished prompts held, to be freed by the call
        return [rng.randint(1, case["most"]) for _ in range(case["rows"])]
    if op == "fork":
        kept = [case["most"] if i == 0 else rng.randint(1, case["most"])
                for i in range(case["sources"])]
        # the rows that the forks replace
        return kept + [rng.randint(1, case["most"]) for _ in range(case["sources"] * case["copies"])]
    live, sizes = max(1, int(case["pages"] * case["live"])), []
    while live > 0:
        n = min(live, rng.randint(1, 64))
        live -= n
        sizes.append(n * case["page"] - rng.randint(0, case["page"] - 1))
    return sizes


def _counts(case):
    """New tokens of each row."""
    n, rng = case["rows"], random.Random(2)
    if not case["prompt"]:
        return [1] * n
    return [case["most"] if i == 0 else rng.randint(1, case["most"]) for i in range(n)]


def _cache(case, g, rng, filled):
    """A cache whose rows hold their tokens on scattered pages; filled: with values."""
    op, kv, d, page = case["op"], case["kv"], case["d"], case["page"]
    layers = case.get("layers", 1)
    sizes = _sizes(case)
    need = [-(-n // page) for n in sizes]
    if op == "compact":
        pages, width = case["pages"], max(need)
    elif op == "append":
        width = -(-(case["most"] + 1) // page)
        pages = case["rows"] * width + 8
    else:
        # forks: the freed rows' pages and one new page each
        width, pages = max(need), sum(need) + 4 + (len(sizes) if op == "fork" else 0)
    numbers = list(range(pages))
    rng.shuffle(numbers)
    table, at = [], 0
    for n in need:
        table.append(numbers[at:at + n] + [-1] * (width - n))
        at += n
    refs = [0] * pages
    for p in numbers[:at]:
        refs[p] = 1
    shape = (layers, pages, kv, page, d)
    c = dict(table=_ints(table), lengths=_ints(sizes), refs=_ints(refs), k_scale=None, v_scale=None)
    for n in ("k", "v"):
        x = torch.zeros(shape, dtype=BF16, device="cuda")
        for layer in range(layers if filled else 0):
            x[layer] = torch.randn(shape[1:], generator=g, device="cuda", dtype=torch.float32).to(BF16)
        if case["bits"] == 8:
            code, scale = torch.empty(shape, dtype=E4M3, device="cuda"), torch.empty(
                shape[:-1], dtype=torch.float32, device="cuda")
            for layer in range(layers):
                code[layer], scale[layer] = _quantise(x[layer])
            c[n], c[n + "_scale"] = code, scale
        else:
            c[n] = x
    return c, sizes


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op, kv, d = case["op"], case["kv"], case["d"]
    s = dict(case=case)
    if op in ("prefill", "backward"):
        ql, kl = _seqs(case)
        H, tq, tk = case["heads"], sum(ql), sum(kl)
        # some queries look sharply, others evenly
        s["q"] = (rand(tq, H, d) * (0.5 + 2.0 * torch.rand(tq, H, 1, generator=g, device="cuda"))).to(BF16)
        s["k"], s["v"] = rand(tk, kv, d).to(BF16), rand(tk, kv, d).to(BF16)
        s["cu_q"], s["cu_k"], s["lens"] = _cu(ql), _cu(kl), (ql, kl)
        if op == "backward":
            s["dout"] = (0.1 * rand(tq, H, d)).to(BF16)
            out, lse = _prefill_plain(s)
            s["out"], s["lse"] = out.to(BF16), lse
        return s
    s["cache"], s["sizes"] = _cache(case, g, rng, op != "append")
    if op == "decode":
        s["q"] = (1.5 * rand(case["rows"], case["heads"], d)).to(BF16)
    elif op == "append":
        n = case["rows"]
        if case["prompt"]:
            counts = _counts(case)
            s["counts"], s["cu"], s["freed"] = _ints(counts), _cu(counts), _ints(list(range(n)))
            s["k"], s["v"] = rand(sum(counts), kv, d).to(BF16), rand(sum(counts), kv, d).to(BF16)
        else:
            # the step's rows have their new token's place already, once for all layers
            s["start"], s["k"], s["v"] = s["cache"]["lengths"] - 1, rand(n, kv, d).to(BF16), \
                rand(n, kv, d).to(BF16)
    elif op == "fork":
        n, m = case["sources"], case["copies"]
        s["src"] = _ints([i for i in range(n) for _ in range(m)])
        s["dst"] = _ints(list(range(n, n + n * m)))
        # the pairs whose source ends inside a page
        s["tails"] = _ints([i for i in range(n * m) if s["sizes"][i // m] % case["page"]]).long()
    else:
        c = s["cache"]
        room = sum(-(-n // case["page"]) for n in s["sizes"]) + 2
        into = {k: None if v is None else torch.zeros((v.shape[0], room, *v.shape[2:]), device="cuda",
                                                      dtype=torch.uint8 if v.dtype == E4M3 else v.dtype)
                for k, v in c.items() if k in ("k", "v", "k_scale", "v_scale")}
        if case["bits"] == 8:
            into["k"], into["v"] = into["k"].view(E4M3), into["v"].view(E4M3)
        s["into"] = dict(into, table=torch.full_like(c["table"], -1), lengths=torch.zeros_like(c["lengths"]),
                         refs=torch.zeros(room, dtype=torch.int32, device="cuda"))
    return s


# -------------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state, state["case"]["op"])


def _whole(c, **more):
    return dict({n: t for n, t in c.items() if t is not None}, **more)


def _run_own(s, op):
    import hybrid_linear_attention_deltanet_gb300 as gdn
    if op == "prefill":
        out, lse = gdn.attention_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
        return dict(out=out, lse=lse)
    if op == "backward":
        return gdn.attention_prefill_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"],
                                              s["cu_q"], s["cu_k"])
    c = s.get("handle")
    if c is None:
        c = s["handle"] = gdn.KVCache(**s["cache"])
    if op == "decode":
        return dict(out=gdn.attention_decode_step(s["q"], c))
    if op == "append":
        start = s.get("start")
        if s["case"]["prompt"]:
            gdn.cache_free(c, s["freed"])
            start = gdn.cache_reserve(c, s["counts"])
        gdn.cache_append(c, s["k"], s["v"], start, s.get("cu"))
        return _whole(s["cache"], start=start)
    if op == "fork":
        gdn.cache_free(c, s["dst"])
        gdn.cache_fork(c, s["src"], s["dst"])
        return _whole(s["cache"])
    if "room" not in s:
        s["room"] = gdn.KVCache(**s["into"])
    gdn.cache_compact(c, s["room"])
    return _whole(s["into"])


def _visible(ql, kl):
    i = torch.arange(ql, device="cuda")[:, None]
    return torch.arange(kl, device="cuda")[None, :] <= i + (kl - ql)


def _prefill_plain(s):
    """out and lse in fp32, sequence by sequence and kv head by kv head."""
    case = s["case"]
    H, kv, d = case["heads"], case["kv"], case["d"]
    G, scale = H // kv, d ** -0.5
    out, lse = torch.zeros(s["q"].shape, device="cuda"), torch.zeros(s["q"].shape[:2], device="cuda")
    a = b = 0
    for ql, kl in zip(*s["lens"]):
        see = _visible(ql, kl)
        for h in range(kv):
            q = s["q"][a:a + ql, h * G:(h + 1) * G].float().transpose(0, 1)
            k, v = s["k"][b:b + kl, h].float(), s["v"][b:b + kl, h].float()
            x = (torch.matmul(q, k.t()) * scale).masked_fill_(~see, -math.inf)
            m = x.amax(-1, keepdim=True)
            x = torch.exp_(x.sub_(torch.where(m == -math.inf, 0.0, m)))
            total = x.sum(-1, keepdim=True)
            o = torch.matmul(x, v) / torch.where(total == 0, 1.0, total)
            out[a:a + ql, h * G:(h + 1) * G] = o.transpose(0, 1)
            lse[a:a + ql, h * G:(h + 1) * G] = (m + torch.log(total))[..., 0].t()
        a, b = a + ql, b + kl
    return out, lse


def _backward_plain(s):
    case = s["case"]
    H, kv, d = case["heads"], case["kv"], case["d"]
    G, scale = H // kv, d ** -0.5
    dq, dk, dv = (torch.zeros(s[n].shape, device="cuda") for n in "qkv")
    a = b = 0
    for ql, kl in zip(*s["lens"]):
        see = _visible(ql, kl)
        for h in range(kv):
            rows, heads = slice(a, a + ql), slice(h * G, (h + 1) * G)
            q, do, o = (s[n][rows, heads].float().transpose(0, 1) for n in ("q", "dout", "out"))
            k, v = s["k"][b:b + kl, h].float(), s["v"][b:b + kl, h].float()
            p = torch.matmul(q, k.t()) * scale
            p = torch.exp_(p.sub_(s["lse"][rows, heads].t()[..., None])).masked_fill_(~see, 0.0)
            dv[b:b + kl, h] = torch.einsum("gij,gid->jd", p, do)
            p.mul_(torch.matmul(do, v.t()).sub_((do * o).sum(-1, keepdim=True)))
            dq[rows, heads] = torch.matmul(p, k).transpose(0, 1) * scale
            dk[b:b + kl, h] = torch.einsum("gij,gid->jd", p, q) * scale
        a, b = a + ql, b + kl
    return dict(dq=dq.to(BF16), dk=dk.to(BF16), dv=dv.to(BF16))


def _decode_plain(s):
    case, c = s["case"], s["cache"]
    H, kv, d, page = case["heads"], case["kv"], case["d"], case["page"]
    out = torch.empty(s["q"].shape, device="cuda")
    for i, n in enumerate(s["sizes"]):
        pages = c["table"][i, :-(-n // page)].long()
        k, v = (c[x][0, pages].float() for x in "kv")
        if case["bits"] == 8:
            k = k * c["k_scale"][0, pages][..., None]
            v = v * c["v_scale"][0, pages][..., None]
        k, v = (t.transpose(0, 1).reshape(kv, -1, d)[:, :n] for t in (k, v))
        x = torch.matmul(s["q"][i].float().view(kv, H // kv, d), k.transpose(1, 2)) * d ** -0.5
        x = torch.exp(x - x.amax(-1, keepdim=True))
        out[i] = (torch.matmul(x, v) / x.sum(-1, keepdim=True)).reshape(H, d)
    return dict(out=out.to(BF16))


def _free_plain(c, rows, page):
    """Every named row gives its pages back."""
    named = torch.zeros(len(c["lengths"]), dtype=torch.bool, device="cuda")
    named[rows.long()] = True
    held = (c["lengths"] + page - 1) // page
    cols = torch.arange(c["table"].shape[1], device="cuda")
    drop = named[:, None] & (cols < held[:, None])
    c["refs"].scatter_add_(0, c["table"].clamp(min=0).flatten().long(), -drop.flatten().int())
    c["table"].masked_fill_(named[:, None], -1)
    c["lengths"].masked_fill_(named, 0)


def _take(c, need):
    """(page numbers in the order they are taken, place of each row's first, which rows get theirs)."""
    free = torch.argsort((c["refs"] != 0).int(), stable=True)
    total = torch.cumsum(need, 0)
    return free, total - need, (need == 0) | (total <= (c["refs"] == 0).sum())


def _reserve_plain(c, counts, page):
    old = (c["lengths"] + page - 1) // page
    new = (c["lengths"] + counts + page - 1) // page
    width = c["table"].shape[1]
    fits = new <= width
    need = torch.where(fits, new - old, 0)
    free, first, ok = _take(c, need)
    ok = ok & fits
    cols = torch.arange(width, device="cuda")
    put = ok[:, None] & (cols >= old[:, None]) & (cols < new[:, None])
    at = (first[:, None] + cols - old[:, None]).clamp(0, len(free) - 1)
    c["table"].copy_(torch.where(put, free[at].int(), c["table"]))
    c["refs"].scatter_add_(0, c["table"].clamp(min=0).flatten().long(), put.flatten().int())
    start = torch.where(ok, c["lengths"], -1)
    c["lengths"].add_(torch.where(ok, counts, 0))
    return start


def _append_plain(s, c, start, page):
    n = len(s["k"])
    at = torch.arange(n, device="cuda")
    row = at if s.get("cu") is None else torch.searchsorted(s["cu"], at, right=True) - 1
    pos = start[row].long() + (0 if s.get("cu") is None else at - s["cu"][row])
    p, slot = c["table"][row, pos // page].long(), pos % page
    for x in "kv":
        if c["k_scale"] is None:
            c[x][0, p, :, slot] = s[x]
        else:
            code, scale = _quantise(s[x])
            c[x].view(torch.uint8)[0, p, :, slot] = code.view(torch.uint8)
            c[x + "_scale"][0, p, :, slot] = scale


def _parts(c):
    """The pools of a cache, 8-bit ones as bytes."""
    return [(n, c[n].view(torch.uint8) if c[n].dtype == E4M3 else c[n])
            for n in ("k", "v", "k_scale", "v_scale") if c[n] is not None]


def _fork_plain(s, c, page):
    src, dst = s["src"].long(), s["dst"].long()
    n = c["lengths"][src]
    full, tail = n // page, n % page
    free, first, _ = _take(c, (tail > 0).int())
    new = free[first.clamp(max=len(free) - 1)].int()
    cols = torch.arange(c["table"].shape[1], device="cuda")
    shared, last = cols < full[:, None], (cols == full[:, None]) & (tail > 0)[:, None]
    old = c["table"][src]
    c["table"][dst] = torch.where(shared, old, torch.where(last, new[:, None], -1))
    c["lengths"][dst] = n
    c["refs"].scatter_add_(0, c["table"][dst].clamp(min=0).flatten().long(),
                           (shared | last).flatten().int())
    was = torch.where(last, old, 0).sum(1).long()
    # the tokens of the last page that are there; what lies behind them stays
    i = s["tails"]
    keep = (torch.arange(page, device="cuda") < tail[i][:, None])[:, None]
    was, to = was[i], new[i].long()
    for _, x in _parts(c):
        for layer in range(x.shape[0]):
            k = keep if x.dim() == 4 else keep[..., None]
            x[layer, to] = torch.where(k, x[layer, was], x[layer, to])


def _compact_plain(c, into, page):
    live = c["refs"] > 0
    name = torch.cumsum(live, 0) - 1
    order = torch.argsort((~live).int(), stable=True)[:len(into["refs"])]
    count = live.sum()
    keep = torch.arange(len(into["refs"]), device="cuda") < count
    pad = len(into["refs"]) - len(order)
    if pad > 0:
        order = torch.cat([order, order.new_zeros(pad)])
    into["refs"].copy_(torch.where(keep, c["refs"][order], 0))
    held = (c["lengths"] + page - 1) // page
    cols = torch.arange(c["table"].shape[1], device="cuda")
    into["table"].copy_(torch.where(cols < held[:, None], name[c["table"].clamp(min=0).long()].int(), -1))
    into["lengths"].copy_(c["lengths"])
    for (_, x), (_, y) in zip(_parts(c), _parts(into)):
        for layer in range(x.shape[0]):
            k = keep.view(-1, *[1] * (x.dim() - 2))
            y[layer] = torch.where(k, x[layer, order], y[layer])


def _run_plain(s, op):
    if op == "prefill":
        out, lse = _prefill_plain(s)
        return dict(out=out.to(BF16), lse=lse)
    if op == "backward":
        return _backward_plain(s)
    if op == "decode":
        return _decode_plain(s)
    c, page = s["cache"], s["case"]["page"]
    if op == "append":
        start = s.get("start")
        if s["case"]["prompt"]:
            _free_plain(c, s["freed"], page)
            start = _reserve_plain(c, s["counts"], page)
        _append_plain(s, c, start, page)
        return _whole(c, start=start)
    if op == "fork":
        _free_plain(c, s["dst"], page)
        _fork_plain(s, c, page)
        return _whole(c)
    _compact_plain(c, s["into"], page)
    return _whole(s["into"])


# ---------------------------------------------------------------- from the definition, 64 bits
def _e4m3_64(v):
    """Nearest e4m3 value of |v| <= 448 in 64 bits, ties to even: 3 fraction bits, exponents
    from -6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _attend_64(q, k, v, shift, scale):
    """Rows q [h, n, d] over keys k, v [h, m, d]; row i sees the keys up to i + shift."""
    x = torch.einsum("hid,hjd->hij", q, k) * scale
    blind = torch.ones(x.shape[1:], dtype=torch.bool, device="cuda").triu(shift + 1)
    x = torch.where(blind, -math.inf, x)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return p, lse, torch.einsum("hij,hjd->hid", p, v)


def _prompts_64(case, s):
    """prefill and backward, a block of query rows at a time, query heads over repeated keys."""
    H, kv, d, B = case["heads"], case["kv"], case["d"], 512
    scale, res = 1.0 / math.sqrt(d), None
    names = ("out", "lse") if case["op"] == "prefill" else ("dq", "dk", "dv")
    like = dict(out=s["q"].shape, lse=s["q"].shape[:2], dq=s["q"].shape, dk=s["k"].shape, dv=s["v"].shape)
    res = {n: torch.zeros(like[n], dtype=torch.float64, device="cuda") for n in names}
    a = b = 0
    for ql, kl in zip(*s["lens"]):
        k, v = (s[n][b:b + kl].double().repeat_interleave(H // kv, 1).transpose(0, 1) for n in "kv")
        for i in range(0, ql, B):
            rows = slice(a + i, a + min(i + B, ql))
            top = max(0, min(kl, min(i + B, ql) + kl - ql))      # keys beyond it: no row sees them
            q = s["q"][rows].double().transpose(0, 1)
            p, lse, o = _attend_64(q, k[:, :top], v[:, :top], i + kl - ql, scale)
            if case["op"] == "prefill":
                res["out"][rows], res["lse"][rows] = o.transpose(0, 1), lse.t()
                continue
            do = s["dout"][rows].double().transpose(0, 1)
            # the given out and lse are the operator's inputs
            p = p * torch.exp(torch.where(lse == -math.inf, 0.0, lse - s["lse"][rows].double().t()))[..., None]
            D = (do * s["out"][rows].double().transpose(0, 1)).sum(-1, keepdim=True)
            ds = p * (torch.einsum("hid,hjd->hij", do, v[:, :top]) - D)
            res["dq"][rows] = scale * torch.einsum("hij,hjd->hid", ds, k[:, :top]).transpose(0, 1)
            for n, w, y in (("dk", ds * scale, q), ("dv", p, do)):
                t = torch.einsum("hij,hid->jhd", w, y)
                res[n][b:b + top] += t.view(top, kv, H // kv, d).sum(2)
        a, b = a + ql, b + kl
    return res


class _Pages:
    """A cache's integers as lists, page by page and row by row."""

    def __init__(self, c, page):
        self.page, self.width = page, c["table"].shape[1]
        self.lengths, self.refs = c["lengths"].tolist(), c["refs"].tolist()
        rows = c["table"].tolist()
        self.rows = [r[:self.held(n)] for r, n in zip(rows, self.lengths)]

    def held(self, n):
        return -(-n // self.page)

    def free(self, rows):
        for r in rows:
            for p in self.rows[r]:
                self.refs[p] -= 1
            self.rows[r], self.lengths[r] = [], 0

    def grow(self, r, n):
        more = self.held(self.lengths[r] + n) - len(self.rows[r])
        got = [p for p, c in enumerate(self.refs) if c == 0][:more]
        assert len(got) == more and len(self.rows[r]) + more <= self.width
        for p in got:
            self.refs[p] = 1
        self.rows[r] += got
        self.lengths[r] += n
        return self.lengths[r] - n

    def tensors(self):
        return dict(table=_ints([r + [-1] * (self.width - len(r)) for r in self.rows]),
                    lengths=_ints(self.lengths), refs=_ints(self.refs))


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("prefill", "backward"):
        return _prompts_64(case, s)
    c, page = s["cache"], case["page"]
    if op == "decode":
        H, kv, d = case["heads"], case["kv"], case["d"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for i, row in enumerate(_Pages(c, page).rows):
            n, pages = s["sizes"][i], torch.tensor(row, device="cuda")
            k, v = (torch.cat(tuple(c[x][0].index_select(0, pages).double() *
                                    (c[x + "_scale"][0].index_select(0, pages).double()[..., None]
                                     if case["bits"] == 8 else 1.0)), 1)[:, :n] for x in "kv")
            q = s["q"][i].double().view(kv, H // kv, d)
            out[i] = _attend_64(q, k, v, n, 1.0 / math.sqrt(d))[2].reshape(H, d)
        return dict(out=out)
    pools = {n: c[n].double() if n.endswith("scale") or op == "append" else c[n].clone()
             for n in ("k", "v", "k_scale", "v_scale") if c[n] is not None}
    pages = _Pages(c, page)
    if op == "append":
        n = case["rows"]
        if case["prompt"]:
            pages.free(range(n))
            start = [pages.grow(r, m) for r, m in enumerate(s["counts"].tolist())]
            counts = s["counts"].tolist()
        else:
            start, counts = s["start"].tolist(), [1] * n
        at = 0
        for r in range(n):
            for p in range(start[r] // page, pages.held(start[r] + counts[r])):
                lo, hi = max(start[r], p * page), min(start[r] + counts[r], (p + 1) * page)
                place = slice(lo - p * page, hi - p * page)
                for x in "kv":
                    t = s[x][at + lo - start[r]:at + hi - start[r]].double().transpose(0, 1)
                    if case["bits"] == 8:
                        m = t.abs().max(-1).values.clamp(min=2.0 ** -100)
                        pools[x + "_scale"][0, pages.rows[r][p], :, place] = m / 448.0
                        t = _e4m3_64(t / m[..., None] * 448.0)
                    pools[x][0, pages.rows[r][p], :, place] = t
            at += counts[r]
        return dict(pools, start=_ints(start), **pages.tensors())
    if op == "fork":
        dst = s["dst"].tolist()
        pages.free(dst)
        for a, b in zip(s["src"].tolist(), dst):
            n = pages.lengths[a]
            whole, tail = n // page, n % page
            pages.rows[b], pages.lengths[b] = pages.rows[a][:whole], whole * page
            for p in pages.rows[b]:
                pages.refs[p] += 1
            if tail:
                pages.grow(b, tail)
                for x in pools.values():
                    x[:, pages.rows[b][-1], :, :tail] = x[:, pages.rows[a][whole], :, :tail]
        return dict(pools, **pages.tensors())
    into = {n: torch.zeros(s["into"][n].shape, dtype=torch.float32 if t.dtype == E4M3 else t.dtype,
                           device="cuda") for n, t in pools.items()}
    kept = [p for p, n in enumerate(pages.refs) if n > 0]
    for new, old in enumerate(kept):
        for n, x in pools.items():
            into[n][:, new] = x[:, old].to(into[n].dtype)
    number = {old: new for new, old in enumerate(kept)}
    pages.refs = [pages.refs[p] for p in kept] + [0] * (len(s["into"]["refs"]) - len(kept))
    pages.rows = [[number[p] for p in r] for r in pages.rows]
    return dict(into, **pages.tensors())


# ------------------------------------------------------------------------------------- work
def work(case):
    op, kv, d = case["op"], case["kv"], case["d"]
    if op in ("prefill", "backward"):
        ql, kl = _seqs(case)
        H, tq, tk = case["heads"], sum(ql), sum(kl)
        pairs = sum(map(_pairs, ql, kl))
        if op == "prefill":
            return dict(bytes=4 * d * (tq * H + tk * kv) + 4 * tq * H, flops=4 * d * H * pairs)
        return dict(bytes=8 * d * (tq * H + tk * kv) + 4 * tq * H, flops=10 * d * H * pairs)
    token = 2 * kv * (d * case["bits"] // 8 + (4 if case["bits"] == 8 else 0))   # k and v, one layer
    if op == "decode":
        tokens = sum(_sizes(case))
        return dict(bytes=tokens * token + 4 * d * case["rows"] * case["heads"],
                    flops=4 * d * case["heads"] * tokens)
    if op == "append":
        tokens = sum(_counts(case))
        return dict(bytes=tokens * (4 * kv * d + token), flops=2 * tokens * kv * d)
    if op == "fork":
        # the last pages' tokens read and written, the tables of the rows
        page, kept = case["page"], _sizes(case)[:case["sources"]]
        tails, table = sum(n % page for n in kept), sum(-(-n // page) for n in kept)
        return dict(bytes=case["copies"] * (2 * case["layers"] * token * tails + 8 * table), flops=0)
    pages = max(1, int(case["pages"] * case["live"]))
    return dict(bytes=2 * pages * case["page"] * case["layers"] * token, flops=0)
