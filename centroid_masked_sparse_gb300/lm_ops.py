"""The operators around the masked head: 4-bit products, attention over an 8-bit cache, token log probabilities.

Thin Python face of the C ABI in include/mtp_lm_ops.h, in the manner of the package's head: each ``mtp_``
function has the name of the C entry point that it calls, takes torch tensors, runs on the current stream (or
``stream``), allocates the outputs that the caller did not pass, and raises ``MtpError`` on a non-OK status.  A call
with a ``stream`` is the call under ``torch.cuda.stream(stream)``: what it allocates belongs to that stream.

    weight = Q4Weight.quantize(w, group=64)                    # once
    logits = mtp_q4_matvec(weight, hidden)                     # [B, M] fp32
    cache = KvCache.allocate(pages, 64, kv_heads, head_dim)
    mtp_kv_append(cache, page_table, lengths, k, v)
    out, lse = mtp_kv_attention(cache, page_table, lengths + 1, q)
    scored = mtp_token_logprobs(logits, tokens, top=5)
    logprob, entropy = token_logprobs(logits, tokens)          # the same, differentiable
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from ._lib import MtpKvBatch, MtpKvDesc, MtpQ4Desc, check, lib

__all__ = ["Q4Weight", "KvCache", "TokenLogprobs", "mtp_q4_quantize", "mtp_q4_matvec", "mtp_kv_append",
           "mtp_kv_attention", "mtp_kv_attention_workspace_bytes", "mtp_token_logprobs",
           "mtp_token_logprobs_backward", "token_logprobs", "MTP_TYPE_F32", "MTP_TYPE_BF16", "MTP_KV_INT8",
           "MTP_KV_E4M3", "MTP_KV_WORKSPACE_ZEROED", "MTP_MAX_TOP", "MTP_DEVERR_PAGE"]

MTP_TYPE_F32, MTP_TYPE_BF16 = 0, 1
MTP_KV_INT8, MTP_KV_E4M3 = 0, 1
MTP_KV_WORKSPACE_ZEROED = 262144
MTP_MAX_TOP = 32
MTP_DEVERR_PAGE = 0x8

_TYPES = {torch.float32: MTP_TYPE_F32, torch.bfloat16: MTP_TYPE_BF16}
_FORMATS = {"int8": MTP_KV_INT8, "e4m3": MTP_KV_E4M3}


# The current stream's handle by device index; torch.cuda.current_stream takes 2 us to wrap it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, index):
    return _raw_stream(index) if stream is None else stream.cuda_stream


# Calls of a few microseconds are all host: the wrappers compare types by identity (there is one object for each)
# and GPUs by number, which take half the time of comparing torch's device objects.
def _vector(t, dtype, n, where):
    """The address of a contiguous tensor of n elements on the call's GPU (get_device()'s number), or None."""
    if t is None:
        return None
    assert t.dtype is dtype and t.numel() == n and t.get_device() == where and t.is_contiguous()
    return t.data_ptr()


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
class Q4Weight:
    """A matrix [M, K] of 4-bit weights, w[m, k] = (code - zero) * scale of its group of columns, packed for
    mtp_q4_matvec when it is made (the tensors that it is made from need not be kept).

    codes    uint8 [M, K / 2]: byte j holds column 2j in its low and 2j + 1 in its high four bits; unit inner
             stride
    scales   bf16 [M, K / group], group 32, 64 or 128
    zeros    uint8 [M, K / group] or None (8 everywhere)
    """

    def __init__(self, codes, scales, zeros=None, stream=None):
        assert codes.is_cuda, "codes must be on a GPU"
        if stream is not None:
            for t in (codes, scales, zeros):
                if t is not None:
                    t.record_stream(stream)   # the caller may drop them before it has packed them
            with torch.cuda.stream(stream):
                return Q4Weight.__init__(self, codes, scales, zeros)
        assert codes.dtype == torch.uint8 and codes.dim() == 2 and codes.stride(1) == 1
        assert scales.dtype == torch.bfloat16 and scales.is_contiguous() and scales.device == codes.device
        assert scales.dim() == 2 and scales.shape[0] == codes.shape[0]
        assert zeros is None or (zeros.dtype == torch.uint8 and zeros.shape == scales.shape and zeros.is_contiguous()
                                 and zeros.device == codes.device)
        self.device, self.index, self.where = codes.device, codes.device.index or 0, codes.get_device()
        self.rows, self.cols = int(codes.shape[0]), 2 * int(codes.shape[1])
        self.group = self.cols // max(1, int(scales.shape[1]))
        assert self.group * int(scales.shape[1]) == self.cols, "scales do not divide the columns into groups"
        size = lib().mtp_q4_packed_bytes(self.rows, self.cols, self.group, zeros is not None)
        self.packed = torch.empty(size, dtype=torch.uint8, device=self.device)
        self.desc = MtpQ4Desc(rows=self.rows, cols=self.cols, group=self.group, zeros=zeros is not None,
                              device=self.index, packed=self.packed.data_ptr(), softcap=0.0)
        check(lib().mtp_q4_pack(ctypes.byref(self.desc), codes.data_ptr(), codes.stride(0) if self.rows > 1 else self.cols // 2,
                                scales.data_ptr(), _ptr(zeros), self.packed.data_ptr(), size, _raw_stream(self.index)),
              "mtp_q4_pack")

    @classmethod
    def quantize(cls, w, group=64, zeros=False, stream=None):
        """The 4-bit form of a bf16 matrix (mtp_q4_quantize), a one-time step."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return cls.quantize(w, group, zeros)
        return cls(*mtp_q4_quantize(w, group, zeros))


def mtp_q4_quantize(w, group=64, zeros=False, stream=None):
    """(codes, scales, zeros or None) of the bf16 matrix w [M, K] (unit inner stride, finite values)."""
    assert w.is_cuda, "w must be on a GPU"
    if stream is not None:
        with torch.cuda.stream(stream):
            return mtp_q4_quantize(w, group, zeros)
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
    rows, cols = w.shape
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(rows, max(1, cols // group), dtype=torch.bfloat16, device=w.device)
    points = torch.empty(scales.shape, dtype=torch.uint8, device=w.device) if zeros else None
    check(lib().mtp_q4_quantize(w.data_ptr(), w.stride(0) if rows > 1 else cols, rows, cols, group, w.device.index or 0,
                                codes.data_ptr(), max(1, cols // 2), scales.data_ptr(), _ptr(points),
                                _raw_stream(w.device.index or 0)), "mtp_q4_quantize")
    return codes, scales, points


def mtp_q4_matvec(weight, x, out=None, out_dtype=torch.float32, softcap=0.0, stream=None):
    """[B, M]: softcap(x @ w.T) of x bf16 [B, K], in fp32 or rounded once to bf16 (out's type, or out_dtype)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mtp_q4_matvec(weight, x, out, out_dtype, softcap)
    batch, cols = x.shape
    rows, where = weight.rows, weight.where
    x_strides = x.stride()
    assert x.dtype is torch.bfloat16 and cols == weight.cols and x_strides[1] == 1 and x.get_device() == where
    if out is None:
        out = torch.empty(batch, rows, dtype=out_dtype, device=weight.device)
    out_strides = out.stride()
    assert out.shape == (batch, rows) and (out_strides[1] == 1 or rows == 1) and out.get_device() == where
    desc = weight.desc
    if softcap != 0.0:
        desc = MtpQ4Desc.from_buffer_copy(desc)
        desc.softcap = softcap
    many = batch > 1
    check(lib().mtp_q4_matvec(desc, x.data_ptr(), x_strides[0] if many else cols, batch, out.data_ptr(), _TYPES[out.dtype],
                              out_strides[0] if many else rows, _raw_stream(weight.index)), "mtp_q4_matvec")
    return out


# ---------------------------------------------------------------------------
# The 8-bit cache
# ---------------------------------------------------------------------------
class KvCache:
    """A paged cache of keys and values in 8 bits, one scale per page and head for each of the two.

    k_codes, v_codes    uint8 [pages, kv_heads, page_tokens, head_dim] contiguous
    k_scales, v_scales  fp32 [pages, kv_heads] contiguous
    format              "int8" or "e4m3"
    """

    def __init__(self, k_codes, v_codes, k_scales, v_scales, format="int8"):
        assert k_codes.is_cuda, "the cache must be on a GPU"
        for t in (k_codes, v_codes):
            assert t.dtype == torch.uint8 and t.dim() == 4 and t.is_contiguous() and t.shape == k_codes.shape
        for t in (k_scales, v_scales):
            assert t.dtype == torch.float32 and t.is_contiguous() and t.shape == k_codes.shape[:2]
        assert len({t.device for t in (k_codes, v_codes, k_scales, v_scales)}) == 1
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.format, self.device, self.index = format, k_codes.device, k_codes.device.index or 0
        self.where = k_codes.get_device()
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = (int(n) for n in k_codes.shape)
        self.errors = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._ws, self._needs = {}, {}   # workspaces by stream, and what calls need by their sizes
        self.desc = MtpKvDesc(num_pages=self.pages, page_tokens=self.page_tokens, kv_heads=self.kv_heads,
                              head_dim=self.head_dim, format=_FORMATS[format], device=self.index,
                              k_codes=k_codes.data_ptr(), v_codes=v_codes.data_ptr(), k_scales=k_scales.data_ptr(),
                              v_scales=v_scales.data_ptr(), error_word=self.errors.data_ptr())

    @classmethod
    def allocate(cls, pages, page_tokens, kv_heads, head_dim, format="int8", device="cuda"):
        """An empty cache (zeros)."""
        def codes():
            return torch.zeros(pages, kv_heads, page_tokens, head_dim, dtype=torch.uint8, device=device)

        def scales():
            return torch.zeros(pages, kv_heads, dtype=torch.float32, device=device)
        return cls(codes(), codes(), scales(), scales(), format)

    def workspace(self, need, stream=None):
        """An attention workspace of at least `need` bytes, zeroed on its stream when it is made.

        One is kept for each stream, since calls on two streams may run at once.  A call that is being captured
        gets one of its own from the graph's memory, with the zeroing in the graph: a kept one may not have been zeroed
        yet when the graph runs, be in use beside it, or make way for a larger one.  Whoever captures can pass a workspace
        (zeroed once, for one graph) to the call and spare the zeroing."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.workspace(need)
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(need, dtype=torch.uint8, device=self.device)
        key = _raw_stream(self.index)
        ws = self._ws.get(key)
        if ws is None or ws.numel() < need:
            ws = self._ws[key] = torch.zeros(need, dtype=torch.uint8, device=self.device)
        return ws

    def read_errors(self):
        """The MTP_DEVERR_* bits that the calls so far have set, on any stream (waits for the GPU), and clears them."""
        torch.cuda.synchronize(self.device)
        bits = int(self.errors.item())
        if bits:
            self.errors.zero_()
            torch.cuda.synchronize(self.device)   # before a call on another stream sets new ones
        return bits


def _token_strides(t, tokens, heads):
    """Strides of tokens and heads, 0 where there is one: tensors carry any number there."""
    token, head, inner = t.stride()
    assert inner == 1
    return token if tokens > 1 else 0, head if heads > 1 else 0


def _batch_desc(cache, page_table, lengths, starts, tokens, max_tokens):
    batch, width = page_table.shape
    where, strides = cache.where, page_table.stride()
    assert page_table.dtype is torch.int32 and page_table.get_device() == where and (strides[1] == 1 or width == 1)
    if max_tokens is None:
        assert starts is None, "ragged calls need the most tokens that one sequence brings"
        max_tokens = max(1, tokens // max(1, batch))
    return MtpKvBatch(batch, tokens, max_tokens, width, page_table.data_ptr(), strides[0] if batch > 1 else width,
                      _vector(lengths, torch.int32, batch, where),
                      None if starts is None else _vector(starts, torch.int32, batch + 1, where))


def mtp_kv_append(cache, page_table, lengths, k, v, starts=None, max_new=None, stream=None) -> None:
    """Write k and v (bf16 [tokens, kv_heads, head_dim]) behind the lengths[b] tokens that each sequence has.

    page_table int32 [B, width], lengths int32 [B]; sequence b brings rows starts[b]..starts[b + 1] (int32
    [B + 1]; at most max_new of them), or without starts an equal share of the rows."""
    shape, where = k.shape, cache.where
    tokens, heads, dim = shape
    assert heads == cache.kv_heads and dim == cache.head_dim and v.shape == shape
    assert k.dtype is torch.bfloat16 and v.dtype is torch.bfloat16 and k.get_device() == where and v.get_device() == where
    k_strides, v_strides = _token_strides(k, tokens, heads), _token_strides(v, tokens, heads)
    seqs = _batch_desc(cache, page_table, lengths, starts, tokens, max_new)
    check(lib().mtp_kv_append(cache.desc, seqs, k.data_ptr(), k_strides[0], k_strides[1],
                              v.data_ptr(), v_strides[0], v_strides[1], _stream(stream, cache.index)), "mtp_kv_append")


def mtp_kv_attention_workspace_bytes(cache, page_table, lengths, tokens, heads, starts=None, max_q=None, max_len=0, window=0) -> int:
    seqs = _batch_desc(cache, page_table, lengths, starts, int(tokens), max_q)
    return int(lib().mtp_kv_attention_workspace_bytes(ctypes.byref(cache.desc), ctypes.byref(seqs), int(heads), int(max_len), int(window)))


def mtp_kv_attention(cache, page_table, lengths, q, starts=None, max_q=None, max_len=0, window=0, scale=None, out=None,
                     lse=None, workspace=None, stream=None):
    """(out bf16 [tokens, heads, head_dim], lse fp32 [tokens, heads]): causal attention of q over the cache.

    lengths are the tokens of each sequence in the cache, with the ones that q belongs to; starts and max_q as
    in mtp_kv_append; max_len bounds the lengths (0: the table's width); window 0 sees everything; scale is
    head_dim ** -0.5 unless given."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mtp_kv_attention(cache, page_table, lengths, q, starts, max_q, max_len, window, scale, out, lse, workspace)
    shape, where = q.shape, cache.where
    tokens, heads, dim = shape
    strides = _token_strides(q, tokens, heads)
    assert q.dtype is torch.bfloat16 and dim == cache.head_dim and q.get_device() == where
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
    if lse is None:
        lse = torch.empty(tokens, heads, dtype=torch.float32, device=cache.device)
    assert out.shape == shape
    seqs = _batch_desc(cache, page_table, lengths, starts, tokens, max_q)
    desc, library = cache.desc, lib()
    if workspace is None:
        # what a call needs goes by its sizes
        key = (seqs.batch, tokens, seqs.max_tokens, seqs.table_width, starts is None, heads, max_len, window)
        need = cache._needs.get(key)
        if need is None:
            if len(cache._needs) > 4096:
                cache._needs.clear()
            need = cache._needs[key] = library.mtp_kv_attention_workspace_bytes(desc, seqs, heads, max_len, window)
        workspace = cache.workspace(need)
    else:
        assert workspace.dtype is torch.uint8 and workspace.get_device() == where and workspace.is_contiguous(), \
            "the workspace must be contiguous bytes on the cache's GPU"
    check(library.mtp_kv_attention(desc, seqs, q.data_ptr(), strides[0], strides[1], heads, max_len, window,
                                   dim ** -0.5 if scale is None else scale, _vector(out, torch.bfloat16, tokens * heads * dim, where),
                                   _vector(lse, torch.float32, tokens * heads, where), workspace.data_ptr(),
                                   workspace.numel(), _raw_stream(cache.index)), "mtp_kv_attention")
    return out, lse


# ---------------------------------------------------------------------------
# Token log probabilities
# ---------------------------------------------------------------------------
class TokenLogprobs(NamedTuple):
    """What mtp_token_logprobs returns, per row: fp32 logprob, entropy and lse, int32 rank, and with top > 0 the
    top_ids (int32) and top_logprobs (fp32) [rows, top]."""
    logprob: torch.Tensor
    entropy: torch.Tensor
    rank: torch.Tensor
    lse: torch.Tensor
    top_ids: Optional[torch.Tensor]
    top_logprobs: Optional[torch.Tensor]


def _rows(t):
    """Rows, columns and row stride of a matrix with unit inner stride."""
    rows, cols = t.shape
    strides = t.stride()
    assert strides[1] == 1 or cols == 1
    return rows, cols, strides[0] if rows > 1 else cols


def mtp_token_logprobs(logits, tokens, top=0, temperature=1.0, out=None, stream=None) -> TokenLogprobs:
    """Log probability and rank of tokens[r] (int32 [rows]; outside the vocabulary: no token) in logits[r], the
    row's entropy and lse, and its `top` largest alternatives.  out: an earlier result to write into."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mtp_token_logprobs(logits, tokens, top, temperature, out)
    rows, vocab, ld = _rows(logits)
    where, kind = logits.get_device(), _TYPES[logits.dtype]
    f32, i32 = torch.float32, torch.int32
    if out is None:
        def empty(*shape, dtype=f32):
            return torch.empty(*shape, dtype=dtype, device=logits.device)
        out = TokenLogprobs(empty(rows), empty(rows), empty(rows, dtype=i32), empty(rows),
                            empty(rows, top, dtype=i32) if top else None, empty(rows, top) if top else None)
    logprob, entropy, rank, lse, top_ids, top_logprobs = out
    check(lib().mtp_token_logprobs(logits.data_ptr(), kind, ld, rows, vocab,
                                   _vector(tokens, i32, rows, where), temperature, top,
                                   _vector(logprob, f32, rows, where), _vector(entropy, f32, rows, where),
                                   _vector(rank, i32, rows, where), _vector(lse, f32, rows, where),
                                   _vector(top_ids, i32, rows * top, where), _vector(top_logprobs, f32, rows * top, where),
                                   where, _raw_stream(where)), "mtp_token_logprobs")
    return out


def mtp_token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob, grad_entropy=None, temperature=1.0, out=None,
                                stream=None):
    """The gradient of sum(grad_logprob * logprob + grad_entropy * entropy) with respect to the logits, in their
    type.  out may be the logits themselves."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mtp_token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob, grad_entropy, temperature, out)
    rows, vocab, ld = _rows(logits)
    where, dtype, f32 = logits.get_device(), logits.dtype, torch.float32
    if out is None:
        out = torch.empty(rows, vocab, dtype=dtype, device=logits.device)
    out_rows, out_cols, ld_out = _rows(out)
    assert out_rows == rows and out_cols == vocab and out.dtype is dtype and out.get_device() == where
    check(lib().mtp_token_logprobs_backward(
        logits.data_ptr(), _TYPES[dtype], ld, rows, vocab, _vector(tokens, torch.int32, rows, where), temperature,
        _vector(lse, f32, rows, where), _vector(entropy, f32, rows, where), _vector(grad_logprob, f32, rows, where),
        _vector(grad_entropy, f32, rows, where), out.data_ptr(), ld_out, where, _raw_stream(where)),
        "mtp_token_logprobs_backward")
    return out


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature):
        scored = mtp_token_logprobs(logits, tokens, temperature=temperature)
        ctx.save_for_backward(logits, tokens, scored.lse, scored.entropy)
        ctx.temperature = temperature
        return scored.logprob, scored.entropy

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_logprob, grad_entropy):
        logits, tokens, lse, entropy = ctx.saved_tensors
        grad = mtp_token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob.contiguous(),
                                           grad_entropy.contiguous(), ctx.temperature)
        return grad, None, None


def token_logprobs(logits, tokens, temperature=1.0):
    """(logprob, entropy), fp32 [rows], differentiable with respect to the logits [rows, vocab] (fp32 or bf16)."""
    return _TokenLogprobs.apply(logits, tokens, temperature)
