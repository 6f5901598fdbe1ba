"""What is measured of the operators around the masked head: 4-bit matrix-vector products, attention over
an 8-bit cache and the append that fills it, and token log probabilities with their gradient.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU, `run()` one pass: in plain torch
operations, or through the package's calls where `own` is true.  `work()` counts what a pass has to move and
compute, `exact()` gives its outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
INT8_MAX, E4M3_MAX = 127.0, 448.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a draft model's projection of one hidden state: latency is all that counts
        dict(name="q4 projection, 1 row", op="q4", rows=2048, cols=1536, group=128, zeros=False, batch=1, out="bf16",
             softcap=0.0),
        # the target's head over the whole vocabulary, verifying eight draft tokens
        dict(name="q4 head, 8 rows", op="q4", rows=262144, cols=1536, group=64, zeros=False, batch=8, out="f32",
             softcap=0.0),
        # an odd vocabulary with zero points, small groups and a softcap, for a ragged verify batch
        dict(name="q4 odd head, 23 rows", op="q4", rows=50021, cols=2592, group=32, zeros=True, batch=23, out="f32",
             softcap=30.0),
        # one user, a long context, one draft token: a single row of queries split over the whole GPU
        dict(name="attend, 1 long sequence", op="attend", batch=1, new=1, heads=8, kv_heads=1, dim=256, page=64,
             longest=65519, window=0, format="int8"),
        # a serving batch of ragged lengths (one of them empty), one token each
        dict(name="attend, 64 ragged", op="attend", batch=64, new=1, heads=32, kv_heads=8, dim=128, page=16,
             longest=8191, window=0, format="e4m3"),
        # verifying up to five tokens a sequence in a sliding-window layer
        dict(name="attend, window, 5 tokens", op="attend", batch=16, new=5, heads=8, kv_heads=4, dim=256, page=32,
             longest=4099, window=512, format="int8"),
        # the step that every decoded token takes: one token a sequence goes into a partly filled block
        dict(name="append, 64 x 1 token", op="append", batch=64, new=1, kv_heads=8, dim=128, page=16, before=1003,
             format="e4m3"),
        # two prompts, the first positions already in the cache
        dict(name="append, 2 x 2049 tokens", op="append", batch=2, new=2049, kv_heads=8, dim=128, page=64, before=37,
             format="e4m3"),
        # one draft row out of the masked head: -inf outside its 4096 candidates, with alternatives
        dict(name="logprobs, 1 masked row", op="logprobs", rows=1, vocab=262144, type="f32", top=5, temperature=1.0,
             candidates=4096),
        # a verify or scoring batch over the whole vocabulary
        dict(name="logprobs, 320 rows", op="logprobs", rows=320, vocab=262144, type="bf16", top=20, temperature=0.7,
             candidates=0),
        # training: the loss's gradient over an odd vocabulary in 32 bits
        dict(name="gradient, 61 odd rows", op="gradient", rows=61, vocab=50021, type="f32", temperature=1.0,
             entropy=False),
        # training a drafter over the whole vocabulary, with an entropy term
        dict(name="gradient, 1024 rows", op="gradient", rows=1024, vocab=262144, type="bf16", temperature=1.0,
             entropy=True),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["q4", "attend", "append", "logprobs", "gradient"])
    if op == "q4":
        group = rng.choice([32, 64, 128])
        cols = group * _log_int(rng, 256 // group, 4096 // group)
        return dict(op=op, rows=_log_int(rng, 256, min(262144, 400_000_000 // cols)), cols=cols, group=group,
                    zeros=rng.random() < 0.5, batch=_log_int(rng, 1, 32), out=rng.choice(["f32", "bf16"]),
                    softcap=rng.choice([0.0, 0.0, 30.0]))
    if op == "attend":
        kv_heads, dim, batch = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, min(65536, 500_000_000 // (batch * kv_heads * dim)))
        return dict(op=op, batch=batch, new=rng.choice([1, 1, 1, 2, 4, 8]), heads=kv_heads * rng.choice([1, 2, 3, 4, 8]),
                    kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]), longest=longest,
                    window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), format=rng.choice(["int8", "e4m3"]))
    if op == "append":
        batch = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, new=_log_int(rng, 1, max(1, 4096 // batch)), kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), before=rng.randint(0, 500),
                    format="e4m3")
    vocab = _log_int(rng, 1000, 262144)
    case = dict(op=op, rows=_log_int(rng, 1, max(1, min(1024, 80_000_000 // vocab))), vocab=vocab,
                type=rng.choice(["f32", "bf16"]), temperature=rng.choice([1.0, 0.7, 1.5]))
    if op == "gradient":
        return dict(case, entropy=rng.random() < 0.5)
    return dict(case, top=rng.choice([0, 1, 5, 20, 32]), candidates=rng.choice([0, 0, vocab // 17]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    return {"q4": _prepare_q4, "attend": _prepare_attend, "append": _prepare_append, "logprobs": _prepare_logprobs,
            "gradient": _prepare_gradient}[case["op"]](case, gen)


def _package():
    import centroid_masked_sparse_gb300
    return centroid_masked_sparse_gb300


def _prepare_q4(case, gen):
    rows, cols, group, batch = case["rows"], case["cols"], case["group"], case["batch"]
    w = torch.randn(rows, cols // group, group, device=DEV, generator=gen) * 0.02
    if case["zeros"]:
        low = w.amin(-1).clamp(max=0)
        scales = ((w.amax(-1).clamp(min=0) - low) / 15).to(torch.bfloat16)
        zeros = (-low / scales.float()).round().clamp(0, 15)
    else:
        scales = (w.abs().amax(-1) / 7).to(torch.bfloat16)
        zeros = torch.full_like(w[..., 0], 8)
    codes = ((w / scales.float()[..., None]).round() + zeros[..., None]).clamp(0, 15).to(torch.uint8).view(rows, cols)
    state = dict(case=case, codes=codes[:, 0::2] | (codes[:, 1::2] << 4), scales=scales,
                 zeros=zeros.to(torch.uint8) if case["zeros"] else None,
                 x=torch.randn(batch, cols, device=DEV, generator=gen).to(torch.bfloat16),
                 out=torch.empty(batch, rows, dtype=_TYPES[case["out"]], device=DEV))
    if own:
        state["weight"] = _package().Q4Weight(state["codes"], state["scales"], state["zeros"])
    return state


def _lengths(case):
    """Tokens of each sequence, the same for every seed: the first is the longest; of several, the last is empty."""
    n, longest = case["batch"], case["longest"]
    lengths = [max(1, round(longest * (0.15 + 0.85 * ((i * 0.6180339887) % 1.0)))) for i in range(n)]
    lengths[0] = longest
    if n > 2:
        lengths[-1] = 0
    return lengths


def _queries(case):
    """Query tokens of each sequence: the full number, fewer in every second one."""
    return [case["new"] if i % 2 == 0 else 1 + i % case["new"] for i in range(case["batch"])]


def _encode(x, scales, fmt):
    x = torch.where(scales > 0, x / scales, 0.0)
    return x.round().to(torch.int8).view(torch.uint8) if fmt == "int8" else x.to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def _largest(fmt):
    return INT8_MAX if fmt == "int8" else E4M3_MAX


def _cache(case, gen, lengths):
    """Page table [B, width] of shuffled pages (-1 beyond a sequence's own) and the pages' codes and scales."""
    page, fmt = case["page"], case["format"]
    need = [-(-n // page) for n in lengths]
    total = sum(need)
    order = torch.randperm(total + 1, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    state = dict(case=case, table=table)
    for name in ("k", "v"):
        x = torch.randn(total + 1, case["kv_heads"], page, case["dim"], device=DEV, generator=gen)
        x *= 0.5 + torch.rand(total + 1, case["kv_heads"], 1, 1, device=DEV, generator=gen)
        scales = x.abs().amax((2, 3)) / _largest(fmt)
        state[name + "_codes"] = _encode(x, scales[..., None, None], fmt)
        state[name + "_scales"] = scales
    if own:
        state["cache"] = _package().KvCache(state["k_codes"], state["v_codes"], state["k_scales"], state["v_scales"], fmt)
    return state


def _prepare_attend(case, gen):
    lengths, queries = _lengths(case), _queries(case)
    state = _cache(case, gen, lengths)
    starts = [0]
    for n in queries:
        starts.append(starts[-1] + n)
    shape = (starts[-1], case["heads"], case["dim"])
    state.update(lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV),
                 starts=torch.tensor(starts, dtype=torch.int32, device=DEV) if case["new"] > 1 else None,
                 q=(torch.randn(*shape, device=DEV, generator=gen) * 1.5).to(torch.bfloat16),
                 out=torch.empty(*shape, dtype=torch.bfloat16, device=DEV),
                 lse=torch.empty(*shape[:2], dtype=torch.float32, device=DEV))
    return state


def _prepare_append(case, gen):
    batch, new, before = case["batch"], case["new"], case["before"]
    state = _cache(case, gen, [before + i % 7 + new for i in range(batch)])
    shape = (batch * new, case["kv_heads"], case["dim"])
    state.update(lengths=torch.tensor([before + i % 7 for i in range(batch)], dtype=torch.int32, device=DEV),
                 k=torch.randn(*shape, device=DEV, generator=gen).to(torch.bfloat16),
                 v=torch.randn(*shape, device=DEV, generator=gen).to(torch.bfloat16))
    return state


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _logits(case, gen):
    rows, vocab = case["rows"], case["vocab"]
    x = (torch.randn(rows, vocab, device=DEV, generator=gen) * 2.5).to(_TYPES[case["type"]])
    given = torch.randint(vocab, (rows,), device=DEV, generator=gen)
    given[::2] = x[::2].argmax(-1)  # what a draft got right
    if case.get("candidates"):
        keep = torch.rand(rows, vocab, device=DEV, generator=gen) < case["candidates"] / vocab
        keep.scatter_(1, given[:, None], True)
        if rows > 4:
            keep[3] = False  # a row whose mask leaves nothing
        x.masked_fill_(~keep, -math.inf)
    if rows > 2:
        given[1] = -1  # a row without a given token
    return dict(case=case, logits=x, tokens=given.to(torch.int32))


def _prepare_logprobs(case, gen):
    state = _logits(case, gen)
    state["out"] = None
    return state


def _prepare_gradient(case, gen):
    state = _logits(case, gen)
    rows = case["rows"]
    x = state["logits"].float() / case["temperature"]
    lse = x.logsumexp(-1)
    x -= lse[:, None]
    state.update(lse=lse, entropy=-(x.exp() * x).sum(-1),
                 grad_logprob=torch.randn(rows, device=DEV, generator=gen) / rows,
                 grad_entropy=torch.randn(rows, device=DEV, generator=gen) / rows if case["entropy"] else None,
                 out=torch.empty_like(state["logits"]))
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return _RUN[state["case"]["op"]][1 if own else 0](state)


def _own_q4(s):
    return _package().mtp_q4_matvec(s["weight"], s["x"], out=s["out"], softcap=s["case"]["softcap"])


def _own_attend(s):
    c = s["case"]
    return _package().mtp_kv_attention(s["cache"], s["table"], s["lengths"], s["q"], starts=s["starts"], max_q=c["new"],
                                       max_len=c["longest"], window=c["window"], out=s["out"], lse=s["lse"])


def _own_append(s):
    _package().mtp_kv_append(s["cache"], s["table"], s["lengths"], s["k"], s["v"])
    return _cache_values(s)


def _own_logprobs(s):
    c = s["case"]
    s["out"] = _package().mtp_token_logprobs(s["logits"], s["tokens"], top=c["top"], temperature=c["temperature"],
                                             out=s["out"])
    return tuple(s["out"])


def _own_gradient(s):
    return _package().mtp_token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], s["grad_logprob"],
                                                  s["grad_entropy"], temperature=s["case"]["temperature"], out=s["out"])


def _cache_values(s):
    """The cache as it stands: its codes as the 8-bit numbers that they are, and the scales."""
    return (s["k_codes"].view(torch.float8_e4m3fn), s["v_codes"].view(torch.float8_e4m3fn), s["k_scales"], s["v_scales"])


def _plain_q4(s):
    case, rows = s["case"], s["case"]["rows"]
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(rows, -1, case["group"]).float()
    codes -= 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    codes *= s["scales"].float()[..., None]
    y = s["x"].float() @ codes.view(rows, -1).T
    if case["softcap"]:
        y = case["softcap"] * torch.tanh(y / case["softcap"])
    return y.to(s["out"].dtype)


def _rows(starts, tokens):
    """Each query token's sequence and its place among that sequence's queries."""
    at = torch.arange(tokens, device=DEV)
    if starts is None:
        return at, torch.zeros_like(at)
    seq = torch.searchsorted(starts[1:].contiguous(), at, right=True)
    return seq, at - starts[seq]


def _plain_attend(s):
    case, table = s["case"], s["table"].clamp(min=0).long()
    batch, new, hkv, dim = case["batch"], case["new"], case["kv_heads"], case["dim"]

    def read(name):
        x = _decode(s[name + "_codes"][table], case["format"]) * s[name + "_scales"][table][..., None, None]
        return x.transpose(1, 2).reshape(batch, hkv, -1, dim)

    tokens = s["q"].shape[0]
    seq, place = _rows(s["starts"], tokens)
    q = torch.zeros(batch, new, hkv, case["heads"] // hkv, dim, device=DEV)
    q[seq, place] = s["q"].float().view(tokens, hkv, -1, dim)
    count = torch.bincount(seq, minlength=batch)
    here = s["lengths"][:, None] - count[:, None] + torch.arange(new, device=DEV)  # [B, new]
    scores = torch.einsum("bqhgd,bhld->bhgql", q, read("k")) / math.sqrt(dim)
    at = torch.arange(scores.shape[-1], device=DEV)
    seen = (at <= here[..., None]) & (at < s["lengths"][:, None, None])
    if case["window"]:
        seen &= at > here[..., None] - case["window"]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgql,bhld->bqhgd", p / torch.where(total == 0, 1.0, total), read("v"))
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)
    return out[seq, place].reshape(tokens, -1, dim).to(torch.bfloat16), lse[seq, place].reshape(tokens, -1)


def _touched(s):
    """The blocks that an append writes: their pages, and of their positions which are new, which old."""
    case, page = s["case"], s["case"]["page"]
    first = s["lengths"] // page
    blocks = first[:, None] + torch.arange((case["new"] + page - 2) // page + 1, device=DEV)  # [B, N]
    at = blocks[..., None] * page + torch.arange(page, device=DEV)  # [B, N, P]
    place = at - s["lengths"][:, None, None]
    new, old = (place >= 0) & (place < case["new"]), place < 0
    real = new.any(-1)
    seq = torch.arange(case["batch"], device=DEV)[:, None].expand_as(blocks)[real]
    row = seq[:, None] * case["new"] + place[real].clamp(0, case["new"] - 1)
    return s["table"][seq, blocks[real]].long(), row, new[real][:, None, :, None], old[real][:, None, :, None]


def _plain_append(s):
    fmt = s["case"]["format"]
    pages, row, new, old = _touched(s)
    for name in ("k", "v"):
        x = s[name][row].float().transpose(1, 2)  # [N, H, P, D]
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        before = torch.where(old.any(2).squeeze(-1), scales[pages], 0.0)
        scale = torch.maximum(before, torch.where(new, x.abs(), 0.0).amax((2, 3)) / _largest(fmt))
        ratio = torch.where(scale > 0, before / scale, 0.0)
        was = codes[pages]
        kept = _encode(_decode(was, fmt) * ratio[..., None, None], torch.ones_like(scale)[..., None, None], fmt)
        codes[pages] = torch.where(new, _encode(x, scale[..., None, None], fmt), torch.where(old, kept, was))
        scales[pages] = scale
    return _cache_values(s)


def _plain_logprobs(s):
    case, raw, given = s["case"], s["logits"], s["tokens"].long()
    vocab = case["vocab"]
    x = raw.float() * (1.0 / case["temperature"])
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    entropy = torch.where(total > 0, torch.log(total) - torch.where(e > 0, e * (x - top), 0.0).sum(-1, keepdim=True) / total, 0.0)
    has = (given >= 0) & (given < vocab)
    at = given.clamp(0, vocab - 1)[:, None]
    mine = x.gather(1, at)
    logprob = torch.where(has[:, None], torch.where(mine == -math.inf, -math.inf, mine - lse), 0.0)
    ids = torch.arange(vocab, device=DEV)
    rank = ((raw > raw.gather(1, at)) | ((raw == raw.gather(1, at)) & (ids < at))).sum(-1)
    outs = [logprob.squeeze(-1), entropy.squeeze(-1), torch.where(has, rank, -1).to(torch.int32), lse.squeeze(-1)]
    if case["top"]:
        bits = (raw.float() + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -2147483649 - bits, bits) * vocab + (vocab - 1 - ids)  # larger first, then the lower id
        best = key.topk(min(case["top"], vocab), dim=-1).indices
        value = x.gather(1, best)
        outs += [torch.where(value == -math.inf, -1, best).to(torch.int32), torch.where(value == -math.inf, -math.inf, value - lse)]
    return tuple(outs)


def _plain_gradient(s):
    case = s["case"]
    given, factor = s["tokens"].long(), 1.0 / case["temperature"]
    has = ((given >= 0) & (given < case["vocab"]))[:, None]
    logp = s["logits"].float() * factor - s["lse"][:, None]
    p = torch.exp(logp)
    weight = torch.where(has, s["grad_logprob"][:, None], 0.0)
    grad = -weight * p
    grad.scatter_add_(1, given.clamp(0, case["vocab"] - 1)[:, None], weight)
    if case["entropy"]:
        grad -= s["grad_entropy"][:, None] * torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0.0)
    return (grad * factor).to(s["logits"].dtype)


_RUN = {"q4": (_plain_q4, _own_q4), "attend": (_plain_attend, _own_attend), "append": (_plain_append, _own_append),
        "logprobs": (_plain_logprobs, _own_logprobs), "gradient": (_plain_gradient, _own_gradient)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "q4":
        groups = case["cols"] // case["group"]
        per_row = case["cols"] // 2 + groups * (3 if case["zeros"] else 2) + case["batch"] * (4 if case["out"] == "f32" else 2)
        return dict(bytes=case["rows"] * per_row + case["batch"] * case["cols"] * 2,
                    flops=2 * case["batch"] * case["rows"] * case["cols"])
    if op == "attend":
        tokens = pairs = 0
        for length, n in zip(_lengths(case), _queries(case)):
            sees = [range(max(0, p - case["window"] + 1) if case["window"] else 0, p + 1) for p in range(length - n, length) if p >= 0]
            pairs += sum(len(r) for r in sees)
            tokens += sees[-1].stop - sees[0].start if sees else 0
        rows = sum(_queries(case))
        return dict(bytes=tokens * case["kv_heads"] * (2 * case["dim"] + 8 / case["page"]) + rows * case["heads"] * (4 * case["dim"] + 4),
                    flops=4 * case["dim"] * case["heads"] * pairs)
    if op == "append":
        values = 2 * case["batch"] * case["new"] * case["kv_heads"] * case["dim"]
        return dict(bytes=values * 3, flops=values * 2)
    values, size = case["rows"] * case["vocab"], 4 if case["type"] == "f32" else 2
    if op == "logprobs":
        return dict(bytes=values * size + case["rows"] * (20 + 8 * case["top"]), flops=values * 6)
    return dict(bytes=values * size * 2 + case["rows"] * 20, flops=values * (7 if case["entropy"] else 4))


# ---------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"q4": _exact_q4, "attend": _exact_attend, "append": _exact_append, "logprobs": _exact_logprobs,
            "gradient": _exact_gradient}[case["op"]](case, s)


def _exact_q4(case, s):
    x, out = s["x"].double(), torch.zeros(case["batch"], case["rows"], dtype=torch.float64, device=DEV)
    for low in range(0, case["rows"], 65536):
        part = slice(low, low + 65536)
        both = s["codes"][part].to(torch.int16)
        w = torch.empty(both.shape[0], case["cols"], dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = both % 16, both // 16
        zero = 8.0 if s["zeros"] is None else s["zeros"][part].double().repeat_interleave(case["group"], 1)
        out[:, part] = x @ ((w - zero) * s["scales"][part].double().repeat_interleave(case["group"], 1)).T
    return case["softcap"] * torch.tanh(out / case["softcap"]) if case["softcap"] else out


def _exact_attend(case, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    row, share = 0, case["heads"] // case["kv_heads"]
    for b, (length, n) in enumerate(zip(_lengths(case), _queries(case))):
        pages = s["table"][b, :-(-length // case["page"])].long()
        k, v = ((_decode(s[c + "_codes"][pages], case["format"]).double() * s[c + "_scales"][pages].double()[:, :, None, None])
                .permute(1, 0, 2, 3).flatten(1, 2)[:, :length].repeat_interleave(share, 0) for c in "kv")
        for i in range(n):
            last = length - n + i + 1
            first = max(0, last - case["window"]) if case["window"] else 0
            if last > first:
                scores = (k[:, first:last] @ s["q"][row + i].double()[:, :, None]).squeeze(-1) / math.sqrt(case["dim"])
                lse[row + i] = scores.logsumexp(-1)
                out[row + i] = (scores.softmax(-1)[:, None] @ v[:, first:last]).squeeze(1)
        row += n
    return out, lse


def _exact_append(case, s):
    page, new, fmt = case["page"], case["new"], case["format"]
    outs = []
    for name in ("k", "v"):
        values, scales = _decode(s[name + "_codes"], fmt).double(), s[name + "_scales"].double()
        for b, before in enumerate(s["lengths"].tolist()):
            x = s[name][b * new:(b + 1) * new].double().transpose(0, 1)  # [H, new, D]
            for block in range(before // page, (before + new - 1) // page + 1):
                at, low, high = int(s["table"][b, block]), max(before, block * page), min(before + new, (block + 1) * page)
                part, first = x[:, low - before:high - before], low - block * page
                was = scales[at] if first else torch.zeros_like(scales[at])
                scale = torch.maximum(was, part.abs().amax((1, 2)) / _largest(fmt))
                values[at, :, :first] *= (was / scale)[:, None, None]
                values[at, :, first:first + high - low] = part / scale[:, None, None]
                scales[at] = scale
        outs.append((values, scales))
    return outs[0][0], outs[1][0], outs[0][1], outs[1][1]


def _exact_logprobs(case, s):
    logprob, entropy, lse, tops = [], [], [], []
    for logits, given in zip(s["logits"].split(64), s["tokens"].long().split(64)):
        x = logits.double() / case["temperature"]
        norm = x.logsumexp(-1, keepdim=True)
        logp = torch.where(x == -math.inf, -math.inf, x - norm)
        mine = logp.gather(1, given.clamp(0, case["vocab"] - 1)[:, None]).squeeze(-1)
        logprob.append(torch.where((given >= 0) & (given < case["vocab"]), mine, 0.0))
        entropy.append(torch.special.entr(logp.exp()).sum(-1))
        lse.append(norm.squeeze(-1))
        if case["top"]:
            tops.append(logp.topk(min(case["top"], case["vocab"]), dim=-1).values)
    outs = (torch.cat(logprob), torch.cat(entropy), None, torch.cat(lse))
    return outs + (None, torch.cat(tops)) if case["top"] else outs


def _exact_gradient(case, s):
    grads = []
    for low in range(0, case["rows"], 64):
        part = slice(low, low + 64)
        given = s["tokens"][part].long()
        logp = torch.log_softmax(s["logits"][part].double() / case["temperature"], -1)
        p = logp.exp()
        has = ((given >= 0) & (given < case["vocab"])).double()
        hot = torch.zeros_like(p).scatter_(1, given.clamp(0, case["vocab"] - 1)[:, None], 1.0)
        grad = (s["grad_logprob"][part].double() * has)[:, None] * (hot - p)
        if case["entropy"]:
            grad -= s["grad_entropy"][part].double()[:, None] * p * (logp - (p * logp).sum(-1, keepdim=True))
        grads.append((grad / case["temperature"]).float() if case["type"] == "bf16" else grad / case["temperature"])
    return torch.cat(grads)
