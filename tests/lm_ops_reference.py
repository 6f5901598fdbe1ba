"""Plain 64-bit forms of the operators around the head, on the CPU, with the error that 32-bit arithmetic allows.

Each function returns the values and, beside them, the largest error that the stated arithmetic may make: the
products of codes and bf16 values are exact in fp32, so what is left is one rounding (2^-24 relative; 2^-23 for
the truncating adds of tensor cores) per addition of a chain, the error of exp2 and log2 (2^-22), one rounding
to bf16 (8 significant bits: 2^-8) where the output has that type, and 2^-11 for the softmax weights, which hold 11 bits.
"""
import math

import torch

U = 2.0 ** -23


def decode(codes, fmt):
    return codes.cpu().view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).double()


def q4_weights(codes, scales, zeros, group):
    codes, scales = codes.cpu(), scales.cpu().double()
    w = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).double()
    zero = torch.full_like(scales, 8.0) if zeros is None else (zeros.cpu() & 15).double()
    return (w - zero.repeat_interleave(group, 1)) * scales.repeat_interleave(group, 1)


def q4_matvec(codes, scales, zeros, group, x, softcap, bf16):
    w, x = q4_weights(codes, scales, zeros, group), x.cpu().double()
    y = x @ w.T
    # chains: 16 products and their sum per tensor step of a group, then the groups, then the parts of a row
    tol = (144 + w.shape[1] / 32) * U * (x.abs() @ w.abs().T)
    if softcap:
        y, tol = softcap * torch.tanh(y / softcap), tol + 8 * U * softcap
    return y, tol + (2.0 ** -8 * (y.abs() + tol) if bf16 else 0.0)


def q4_quantize(w, group, zeros):
    """codes, scales, zeros: the definition in fp32, step by step (exact comparison)."""
    w = w.cpu().float().view(w.shape[0], -1, group)
    if zeros:
        low, high = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        scales = ((high - low) / 15).to(torch.bfloat16)
        points = torch.where(scales > 0, -low / scales.float(), 0.0).round().clamp(0, 15)
    else:
        scales = (w.abs().amax(-1) / 7).to(torch.bfloat16)
        points = torch.full(scales.shape, 8.0)
    s = scales.float()[..., None]
    codes = (torch.where(s > 0, w / s, 0.0).round() + points[..., None]).clamp(0, 15).to(torch.uint8).flatten(1)
    return codes[:, 0::2] | codes[:, 1::2] << 4, scales, points.to(torch.uint8) if zeros else None


def attention(q, k_codes, v_codes, k_scales, v_scales, fmt, table, lengths, starts, window, scale):
    """(out, its error, lse, its error); rows that no sequence brings are NaN."""
    q, table = q.cpu().double(), table.cpu().long()
    heads, dim = q.shape[1:]
    share, page = heads // k_codes.shape[1], k_codes.shape[2]
    ks, vs = k_scales.cpu().double(), v_scales.cpu().double()
    outs = [torch.full(q.shape, math.nan, dtype=torch.float64) for _ in range(2)]
    lses = [torch.full(q.shape[:2], math.nan, dtype=torch.float64) for _ in range(2)]
    for b, length in enumerate(lengths):
        pages = table[b, :-(-length // page)]
        read = []
        for codes, scales in ((k_codes, ks), (v_codes, vs)):
            x = decode(codes[pages.to(codes.device)], fmt) * scales[pages][:, :, None, None]
            read.append(x.transpose(0, 1).flatten(1, 2)[:, :length].repeat_interleave(share, 0))
        k, v = read
        n = starts[b + 1] - starts[b]
        for i in range(n):
            row, here = starts[b] + i, length - n + i
            low = max(0, here - window + 1) if window else 0
            if here < 0:
                outs[0][row], outs[1][row], lses[0][row], lses[1][row] = 0, 0, -math.inf, 0
                continue
            kk, vv, qq = k[:, low:here + 1], v[:, low:here + 1], q[row][:, None]
            s = scale * (kk * qq).sum(-1)
            most = abs(scale) * (kk * qq).abs().sum(-1).amax(-1)                     # [heads]
            ds = (dim + 8) * U * most + 2.0 ** -21 * (1 + s.abs().amax(-1))           # scores, exp2
            p = s.softmax(-1)
            o, size = (p[..., None] * vv).sum(1), (p[..., None] * vv.abs()).sum(1)
            count = here + 1 - low
            chain = (64 + count / 16) * U
            outs[0][row] = o
            outs[1][row] = (2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * ds + 2 * chain)[:, None] * size
                            + count * 2.0 ** -25 * vv.abs().amax(1) * p.amax(-1)[:, None])
            lses[0][row] = s.logsumexp(-1)
            lses[1][row] = ds + chain + 4 * U * lses[0][row].abs()
    return outs[0], outs[1], lses[0], lses[1]


def append(k_codes, scales, fmt, table, lengths, starts, x):
    """The cache's codes and scales (one of keys and values) after the append, in fp32 as it is defined."""
    codes, scales, x = k_codes.cpu().clone(), scales.cpu().clone(), x.cpu().float()
    x = torch.nan_to_num(x, nan=0.0, posinf=3.3895313892515355e38, neginf=-3.3895313892515355e38)
    page, most = codes.shape[2], torch.tensor(127.0 if fmt == "int8" else 448.0)
    view = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)

    def encode(v):
        return v.round().to(torch.int8) if fmt == "int8" else v.to(torch.float8_e4m3fn)

    for b, before in enumerate(lengths):
        n = starts[b + 1] - starts[b]
        for block in range(before // page, (before + n - 1) // page + 1 if n else 0):
            at = int(table[b, block])
            low, high = max(before, block * page), min(before + n, (block + 1) * page)
            part = x[starts[b] + low - before:starts[b] + high - before].transpose(0, 1)
            first = low - block * page
            was = scales[at] if first else torch.zeros_like(scales[at])
            scale = torch.maximum(was, part.abs().amax((1, 2)) / most)
            safe = torch.where(scale > 0, scale, 1.0)[:, None, None]
            ratio = torch.where(scale > 0, was / safe[:, 0, 0], 0.0)[:, None, None]
            view[at, :, :first] = encode(view[at, :, :first].float() * ratio)
            view[at, :, first:first + high - low] = encode(torch.where(scale[:, None, None] > 0, part / safe, 0.0))
            scales[at] = scale
    return codes, scales


def logprobs(logits, tokens, temperature, top):
    """Values and errors: dict of name -> (value, error); errors 0 where the value is exact."""
    raw, given = logits.cpu(), tokens.cpu().long()
    rows, vocab = raw.shape
    x = raw.double() / float(torch.tensor(temperature))
    lse = x.logsumexp(-1)
    logp = torch.where(x == -math.inf, -math.inf, x - lse[:, None])
    p = logp.exp()
    has = (given >= 0) & (given < vocab)
    at = given.clamp(0, vocab - 1)[:, None]
    mine = torch.where(has, logp.gather(1, at).squeeze(1), 0.0)
    r = raw.float() + 0.0
    y, ids = r.gather(1, at), torch.arange(vocab)
    rank = torch.where(has, ((r > y) | ((r == y) & (ids < at))).sum(-1), -1)
    # one rounding of x c - m per term, three of the statistics, and the terms' sum
    size = torch.nan_to_num(x.amax(-1), neginf=0.0).abs() + math.log(vocab) + 8
    tol = 2.0 ** -22 * size + vocab / 256 * 2.0 ** -24
    spread = torch.where(p > 0, p * logp.abs(), 0.0).sum(-1)
    out = dict(logprob=(mine, torch.where(mine == -math.inf, 0.0, tol + 2.0 ** -22 * torch.nan_to_num(mine, neginf=0.0).abs())),
               entropy=(torch.special.entr(p).sum(-1), tol * (2 + spread)), rank=(rank, None), lse=(lse, tol))
    if top:
        order = (-r.double()).sort(dim=-1, stable=True).indices[:, :top]
        value = logp.gather(1, order)
        ids = torch.where(value == -math.inf, -1, order)
        pad = top - order.shape[1]
        ids = torch.nn.functional.pad(ids, (0, pad), value=-1)
        value = torch.nn.functional.pad(value, (0, pad), value=-math.inf)
        out.update(top_ids=(ids, None), top_logprobs=(value, tol[:, None] + 2.0 ** -22 * torch.nan_to_num(value, neginf=0.0).abs()))
    return out


def logprobs_grad(logits, tokens, temperature, grad_logprob, grad_entropy, bf16):
    raw, given, t = logits.cpu(), tokens.cpu().long(), float(torch.tensor(temperature))
    vocab = raw.shape[1]
    x = raw.double() / t
    lse = x.logsumexp(-1, keepdim=True)
    logp = torch.where(x == -math.inf, -math.inf, x - lse)
    p = logp.exp()
    safe = torch.where(p > 0, logp, 0.0)
    entropy = torch.special.entr(p).sum(-1, keepdim=True)
    has = ((given >= 0) & (given < vocab)).double()
    hot = torch.zeros_like(p).scatter_(1, given.clamp(0, vocab - 1)[:, None], has[:, None])
    gl = (torch.zeros_like(has) if grad_logprob is None else grad_logprob.cpu().double() * has)[:, None]
    ge = torch.zeros_like(gl) if grad_entropy is None else grad_entropy.cpu().double()[:, None]
    live = (x > -math.inf).double()
    grad = (gl * (hot - p) - ge * p * (safe + entropy)) / t * live
    off = 2.0 ** -22 * (torch.nan_to_num(lse, neginf=0.0).abs() + torch.nan_to_num(x, neginf=0.0).abs() + 16)  # of ln p, and of lse
    size = (gl.abs() * (hot + p) + ge.abs() * p * (safe.abs() + entropy + 1)) / t
    tol = off * size + 8 * U * size + vocab / 256 * 2.0 ** -24 * size
    return grad, tol + (2.0 ** -8 * grad.abs() if bf16 else 0.0) + 1e-37
