"""The refusals of the operators around the head: host-side checks, which launch nothing."""
import ctypes

import pytest

NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -3, -4, -6


@pytest.fixture(scope="module")
def L():
    from centroid_masked_sparse_gb300 import build
    build.build()
    from centroid_masked_sparse_gb300 import _lib
    return _lib.lib()


def q4(**kw):
    from centroid_masked_sparse_gb300._lib import MtpQ4Desc
    return MtpQ4Desc(**{**dict(rows=100, cols=256, group=64, zeros=0, device=0, packed=0x1000, softcap=0.0), **kw})


Q4_REFUSALS = [(dict(rows=0), {}, SHAPE), (dict(cols=0), {}, SHAPE), (dict(cols=250), {}, SHAPE), (dict(group=16), {}, UNSUPPORTED),
               (dict(group=128, cols=192), {}, SHAPE), (dict(cols=16384 + 64), {}, UNSUPPORTED), (dict(device=-1), {}, SHAPE)]


@pytest.mark.parametrize("desc,call,expect", Q4_REFUSALS + [
    (dict(packed=None), {}, NULL), (dict(packed=0x1080), {}, ALIGN),
    (dict(softcap=-1.0), {}, SHAPE), (dict(softcap=float("nan")), {}, SHAPE),
    ({}, dict(x=None), NULL), ({}, dict(out=None), NULL), ({}, dict(x=0x3004), ALIGN), ({}, dict(ld_x=255), SHAPE),
    ({}, dict(ld_x=260), ALIGN), ({}, dict(ld_out=99), SHAPE), ({}, dict(out=0x4002), ALIGN), ({}, dict(batch=-1), SHAPE),
    ({}, dict(batch=1025), UNSUPPORTED), ({}, dict(out_type=2), UNSUPPORTED), ({}, dict(batch=0, x=None, out=None), 0),
])
def test_q4_matvec_refuses(L, desc, call, expect):
    c = {**dict(x=0x3000, ld_x=256, batch=4, out=0x4000, out_type=0, ld_out=100), **call}
    assert L.mtp_q4_matvec(ctypes.byref(q4(**desc)), c["x"], c["ld_x"], c["batch"], c["out"], c["out_type"], c["ld_out"],
                           None) == expect


@pytest.mark.parametrize("desc,call,expect", Q4_REFUSALS + [
    ({}, dict(codes=None), NULL), ({}, dict(scales=None), NULL), ({}, dict(packed=None), NULL), ({}, dict(zeros=0x7000), NULL),
    (dict(zeros=1), {}, NULL), ({}, dict(ld=127), SHAPE), ({}, dict(size=1000), SHAPE), ({}, dict(scales=0x3001), ALIGN),
    ({}, dict(packed=0x4010), ALIGN),
])
def test_q4_pack_refuses(L, desc, call, expect):
    c = {**dict(codes=0x2001, ld=128, scales=0x3000, zeros=None, packed=0x4000, size=1 << 30), **call}
    assert L.mtp_q4_pack(ctypes.byref(q4(**desc)), c["codes"], c["ld"], c["scales"], c["zeros"], c["packed"], c["size"],
                         None) == expect


def test_q4_packed_bytes(L):
    # 7 tiles of 16 rows: 4 blocks of 512 bytes, 1 step of 8 x 4 x 2 scales of 2 bytes
    assert L.mtp_q4_packed_bytes(100, 256, 64, 0) == 7 * 4 * 512 + (7 * 128 + 255) // 256 * 256
    assert L.mtp_q4_packed_bytes(100, 256, 64, 1) == L.mtp_q4_packed_bytes(100, 256, 64, 0) + (7 * 64 + 255) // 256 * 256
    assert L.mtp_q4_packed_bytes(100, 250, 64, 0) == 0 and L.mtp_q4_packed_bytes(0, 256, 64, 0) == 0


def test_q4_matvec_refuses_no_descriptor(L):
    assert L.mtp_q4_matvec(None, 0x3000, 256, 4, 0x4000, 0, 100, None) == NULL


@pytest.mark.parametrize("kw,expect", [
    (dict(w=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(rows=0), SHAPE), (dict(group=48), UNSUPPORTED),
    (dict(cols=100), SHAPE), (dict(ld_w=200), SHAPE), (dict(ld_codes=100), SHAPE), (dict(w=0x1001), ALIGN),
])
def test_q4_quantize_refuses(L, kw, expect):
    c = {**dict(w=0x1000, ld_w=256, rows=4, cols=256, group=64, codes=0x2000, ld_codes=128, scales=0x3000), **kw}
    assert L.mtp_q4_quantize(c["w"], c["ld_w"], c["rows"], c["cols"], c["group"], 0, c["codes"], c["ld_codes"], c["scales"], None,
                             None) == expect


def kv(**kw):
    from centroid_masked_sparse_gb300._lib import MtpKvDesc
    return MtpKvDesc(**{**dict(num_pages=10, page_tokens=32, kv_heads=2, head_dim=128, format=0, device=0, k_codes=0x10000,
                               v_codes=0x20000, k_scales=0x30000, v_scales=0x40000, error_word=None), **kw})


def seqs(**kw):
    from centroid_masked_sparse_gb300._lib import MtpKvBatch
    return MtpKvBatch(**{**dict(batch=2, tokens=2, max_tokens=1, table_width=4, page_table=0x50000, ld_table=4, lengths=0x60000,
                                starts=None), **kw})


CACHE_REFUSALS = [
    (dict(num_pages=0), {}, SHAPE), (dict(kv_heads=0), {}, SHAPE), (dict(page_tokens=8), {}, SHAPE), (dict(page_tokens=40), {}, SHAPE),
    (dict(page_tokens=2048), {}, UNSUPPORTED), (dict(kv_heads=2000), {}, UNSUPPORTED), (dict(head_dim=96), {}, UNSUPPORTED),
    (dict(format=2), {}, UNSUPPORTED), (dict(device=-1), {}, SHAPE), (dict(k_codes=None), {}, NULL), (dict(v_codes=None), {}, NULL),
    (dict(k_scales=None), {}, NULL), (dict(v_scales=None), {}, NULL), (dict(k_codes=0x10008), {}, ALIGN),
    (dict(v_scales=0x40002), {}, ALIGN), (dict(error_word=0x70001), {}, ALIGN), ({}, dict(batch=-1), SHAPE),
    ({}, dict(tokens=-1), SHAPE), ({}, dict(batch=70000, tokens=70000), UNSUPPORTED), ({}, dict(page_table=None), NULL),
    ({}, dict(lengths=None), NULL), ({}, dict(max_tokens=0), SHAPE), ({}, dict(table_width=0), SHAPE), ({}, dict(ld_table=3), SHAPE),
    ({}, dict(tokens=3), SHAPE), ({}, dict(starts=0x70002, tokens=3), ALIGN),
]


@pytest.mark.parametrize("desc,batch,call,expect", [(*r[:2], {}, r[2]) for r in CACHE_REFUSALS] + [
    ({}, {}, dict(k=None), NULL), ({}, {}, dict(v=None), NULL), ({}, {}, dict(k=0x80008), ALIGN), ({}, {}, dict(token=100), ALIGN),
    ({}, {}, dict(head=4), ALIGN), ({}, {}, dict(token=-8), SHAPE), ({}, dict(batch=0, tokens=0), dict(k=None), 0),
    ({}, dict(tokens=0), dict(k=None), 0),
])
def test_kv_append_refuses(L, desc, batch, call, expect):
    c = {**dict(k=0x80000, v=0x90000, token=256, head=128), **call}
    assert L.mtp_kv_append(ctypes.byref(kv(**desc)), ctypes.byref(seqs(**batch)), c["k"], c["token"], c["head"], c["v"], 256, 128,
                           None) == expect


@pytest.mark.parametrize("desc,batch,call,expect", [(*r[:2], {}, r[2]) for r in CACHE_REFUSALS] + [
    ({}, {}, dict(heads=0), SHAPE), ({}, {}, dict(heads=5), SHAPE), ({}, {}, dict(heads=65536 * 2), UNSUPPORTED),
    ({}, {}, dict(max_len=-1), SHAPE), ({}, {}, dict(window=-1), SHAPE), ({}, {}, dict(q=None), NULL), ({}, {}, dict(q=0x80004), ALIGN),
    ({}, {}, dict(token=1001), ALIGN), ({}, {}, dict(head=-8), SHAPE), ({}, {}, dict(out=None), NULL), ({}, {}, dict(out=0x90008), ALIGN),
    ({}, {}, dict(lse=0xa0002), ALIGN), ({}, {}, dict(ws=None), WORKSPACE), ({}, {}, dict(ws_bytes=1000), WORKSPACE),
    ({}, {}, dict(ws=0xb0004), ALIGN), ({}, dict(tokens=0), dict(q=None, out=None, ws=None), 0),
])
def test_kv_attention_refuses(L, desc, batch, call, expect):
    c = {**dict(q=0x80000, token=1024, head=128, heads=8, max_len=0, window=0, out=0x90000, lse=None, ws=0xb0000, ws_bytes=1 << 40),
         **call}
    assert L.mtp_kv_attention(ctypes.byref(kv(**desc)), ctypes.byref(seqs(**batch)), c["q"], c["token"], c["head"], c["heads"],
                              c["max_len"], c["window"], 0.1, c["out"], c["lse"], c["ws"], c["ws_bytes"], None) == expect


def test_kv_attention_refuses_no_descriptor(L):
    assert L.mtp_kv_attention(None, ctypes.byref(seqs()), 0x80000, 1024, 128, 8, 0, 0, 0.1, 0x90000, None, 0xb0000, 1 << 40, None) == NULL
    assert L.mtp_kv_append(ctypes.byref(kv()), None, 0x80000, 256, 128, 0x90000, 256, 128, None) == NULL


def test_kv_attention_workspace(L):
    from centroid_masked_sparse_gb300 import MTP_KV_WORKSPACE_ZEROED
    need = L.mtp_kv_attention_workspace_bytes(ctypes.byref(kv()), ctypes.byref(seqs()), 8, 0, 0)
    assert need >= MTP_KV_WORKSPACE_ZEROED
    assert L.mtp_kv_attention_workspace_bytes(ctypes.byref(kv()), ctypes.byref(seqs()), 5, 0, 0) == 0
    assert L.mtp_kv_attention_workspace_bytes(ctypes.byref(kv(head_dim=80)), ctypes.byref(seqs()), 8, 0, 0) == 0
    assert L.mtp_kv_attention_workspace_bytes(ctypes.byref(kv()), ctypes.byref(seqs()), 8, -1, 0) == 0


def test_kv_attention_limits(L):
    """Caches of more than 2^30 tokens a sequence and calls of more than 2^19 query rows are refused; workspaces follow
    the split of every kind of call and are refused when they are short."""
    def call(batch, heads=8, window=0, ws_bytes=1 << 40):
        return L.mtp_kv_attention(ctypes.byref(kv()), ctypes.byref(batch), 0x80000, 1 << 20, 128, heads, 0, window, 0.1, 0x90000, None,
                                  0xb0000, ws_bytes, None)
    assert call(seqs(table_width=(1 << 25) + 1, ld_table=(1 << 25) + 1)) == UNSUPPORTED
    assert call(seqs(batch=1, tokens=(1 << 16) + 1, max_tokens=(1 << 16) + 1)) == UNSUPPORTED
    assert call(seqs(), heads=65536) == UNSUPPORTED
    for batch in (seqs(batch=1, tokens=1, table_width=4096, ld_table=4096), seqs(batch=64, tokens=64), seqs(batch=3, tokens=9, max_tokens=7)):
        for window in (0, 1, 100):
            for max_len in (0, 1, 1 << 30):
                assert L.mtp_kv_attention_workspace_bytes(ctypes.byref(kv()), ctypes.byref(batch), 8, max_len, window) >= 262144
            assert call(batch, window=window, ws_bytes=262143) == WORKSPACE


@pytest.mark.parametrize("kw,expect", [
    (dict(type=2), UNSUPPORTED), (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(ld=999), SHAPE), (dict(temperature=0.0), SHAPE),
    (dict(temperature=-1.0), SHAPE), (dict(temperature=float("nan")), SHAPE), (dict(temperature=float("inf")), SHAPE),
    (dict(top=-1), SHAPE), (dict(top=33), UNSUPPORTED), (dict(logits=None), NULL), (dict(tokens=None), NULL), (dict(ids=None, top=1), NULL),
    (dict(logits=0x1002), ALIGN), (dict(tokens=0x2002), ALIGN), (dict(logprob=0x3001), ALIGN), (dict(device=-1), SHAPE),
    (dict(rows=0, logits=None, tokens=None), 0),
])
def test_token_logprobs_refuses(L, kw, expect):
    c = {**dict(logits=0x1000, type=0, ld=1000, rows=3, vocab=1000, tokens=0x2000, temperature=1.0, top=0, logprob=0x3000, ids=0x4000,
                device=0), **kw}
    assert L.mtp_token_logprobs(c["logits"], c["type"], c["ld"], c["rows"], c["vocab"], c["tokens"], c["temperature"], c["top"],
                                c["logprob"], None, None, None, c["ids"], None, c["device"], None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(type=3), UNSUPPORTED), (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(ld=999), SHAPE), (dict(ld_grad=999), SHAPE),
    (dict(temperature=0.0), SHAPE), (dict(logits=None), NULL), (dict(lse=None), NULL), (dict(grad=None), NULL), (dict(gl=None), NULL),
    (dict(tokens=None), NULL), (dict(ge=0x7000, entropy=None), NULL), (dict(grad=0x1000, ld_grad=1001), SHAPE), (dict(grad=0x5002), ALIGN),
    (dict(lse=0x4001), ALIGN), (dict(rows=0, logits=None), 0),
])
def test_token_logprobs_backward_refuses(L, kw, expect):
    c = {**dict(logits=0x1000, type=0, ld=1000, rows=3, vocab=1000, tokens=0x2000, temperature=1.0, lse=0x4000, entropy=0x4100,
                gl=0x4200, ge=None, grad=0x5000, ld_grad=1000), **kw}
    assert L.mtp_token_logprobs_backward(c["logits"], c["type"], c["ld"], c["rows"], c["vocab"], c["tokens"], c["temperature"], c["lse"],
                                         c["entropy"], c["gl"], c["ge"], c["grad"], c["ld_grad"], 0, None) == expect


def test_kv_bound_above_the_tokens_counts_as_the_tokens(L):
    """A capacity as the most tokens of a sequence neither makes a call too large nor its workspace larger."""
    ragged = dict(batch=2, tokens=5, starts=0x70000, table_width=4096, ld_table=4096)
    need = [L.mtp_kv_attention_workspace_bytes(ctypes.byref(kv()), ctypes.byref(seqs(max_tokens=n, **ragged)), 8, 0, 0)
            for n in (5, 100, 1 << 20, (1 << 31) - 1)]
    assert len(set(need)) == 1
    for n in (5, 1 << 20, (1 << 31) - 1):
        # short of the workspace, which is looked at after the sizes
        assert L.mtp_kv_attention(ctypes.byref(kv()), ctypes.byref(seqs(max_tokens=n, **ragged)), 0x80000, 1024, 128, 8, 0, 0, 0.1,
                                  0x90000, None, 0xb0000, 1000, None) == WORKSPACE


def test_temperatures_whose_factor_leaves_the_range_are_refused(L):
    for temperature, refused in ((3.2e-39, True), (4.1e-39, True), (4.4e-39, False), (1e-38, False)):
        # a bad output address is looked at after the temperature
        status = [L.mtp_token_logprobs(0x1000, 0, 1000, 3, 1000, 0x2000, temperature, 0, 0x3001, None, None, None, None, None, 0, None),
                  L.mtp_token_logprobs_backward(0x1000, 0, 1000, 3, 1000, 0x2000, temperature, 0x4001, None, 0x4200, None, 0x5000, 1000, 0,
                                                None)]
        assert status == [SHAPE if refused else ALIGN] * 2
