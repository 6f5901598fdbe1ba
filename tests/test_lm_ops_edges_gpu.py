"""The operators around the head on the GPU at the ends of their ranges: magnitudes, temperatures, lengths, bounds,
strides, streams and what a query must not see, against 64-bit forms."""
import math

import pytest

torch = pytest.importorskip("torch")

import centroid_masked_sparse_gb300 as mtp
from tests import lm_ops_reference as ref
from tests.test_lm_ops_gpu import BF16, DEV, F32, close, gen, ints, make_cache, q4_weight, randn

pytestmark = pytest.mark.gpu
U = ref.U


def exact_gradient(logits, tokens, temperature, gl, ge):
    raw, given = logits.cpu().double(), tokens.cpu().long()
    vocab, t = raw.shape[1], float(torch.tensor(temperature))
    top = raw.amax(-1, keepdim=True)
    d = torch.where(raw == -math.inf, -math.inf, (raw - torch.nan_to_num(top, neginf=0.0)) / t)
    lse0 = d.logsumexp(-1, keepdim=True)
    logp = torch.where(raw == -math.inf, -math.inf, d - lse0)
    p = logp.exp()
    safe = torch.where(p > 0, logp, 0.0)
    h = torch.special.entr(p).sum(-1, keepdim=True)
    has = ((given >= 0) & (given < vocab)).double()[:, None]
    hot = torch.zeros_like(p).scatter_(1, given.clamp(0, vocab - 1)[:, None], has)
    gl = torch.zeros_like(has) if gl is None else gl.cpu().double()[:, None] * has
    ge = torch.zeros_like(has) if ge is None else ge.cpu().double()[:, None]
    live = (raw > -math.inf).double()
    grad = (gl * (hot - p) - ge * p * (safe + h)) / t * live
    lse = (top / t + lse0).abs()
    off = 2.0 ** -24 * torch.where(lse < 1024, lse, 0.0) + 2.0 ** -22 * (16 + safe.abs().clamp(max=200))
    size = (gl.abs() * (hot * live + p) + ge.abs() * p * (safe.abs() + h + 1)) / t
    return grad, (off + 8 * U + vocab / 256 * 2.0 ** -24) * size


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 8.0])
@pytest.mark.parametrize("vocab", [37, 5003, 40000])
def test_gradient_of_rows_of_large_magnitude(dtype, temperature, vocab):
    """Rows where the fp32 lse leaves no room for ln V, and the type's lowest value as a mask, of some tokens or all."""
    g = gen(vocab)
    lowest = torch.finfo(dtype).min * 0.5 if temperature < 1 else torch.finfo(dtype).min
    logits = randn(g, 12, vocab).to(dtype)
    logits[0] = lowest
    logits[1] = lowest
    logits[1, vocab // 2] = 3.0
    logits[2] = -1e9
    logits[3] = 1e9
    logits[4] -= 2000
    logits[5] = logits[5] * 4 + 30000
    logits[6] = logits[6] * 1e6
    logits[7] = -1e9
    logits[7, ::3] = -math.inf
    logits[8] = -1e30
    logits[8, 5:11] = randn(g, 6).to(dtype)
    logits[9] += 700
    logits[10] = lowest
    logits[10, 1::2] = -math.inf
    tokens = torch.randint(vocab, (12,), device=DEV, generator=g).to(torch.int32)
    for given in (tokens, torch.full_like(tokens, -1)):
        fw = mtp.mtp_token_logprobs(logits, given, temperature=temperature)
        for gl, ge in ((randn(g, 12), randn(g, 12)), (randn(g, 12), None), (None, randn(g, 12))):
            got = mtp.mtp_token_logprobs_backward(logits, given, fw.lse, fw.entropy, gl, ge, temperature)
            want, tol = exact_gradient(logits, given, temperature, gl, ge)
            close(got, want, tol + (2.0 ** -8 * want.abs() if dtype == BF16 else 0.0) + 1e-37, f"{gl is None} {ge is None}")


def test_gradient_of_masked_tokens_with_large_weights():
    """A token without weight gets 0, not 0 times an overflow, however large the entropy's weight is."""
    g = gen(41)
    logits = randn(g, 4, 1000)
    logits[:, ::2] = -math.inf
    tokens = ints([1, 3, 5, 7])
    fw = mtp.mtp_token_logprobs(logits, tokens, temperature=1e-3)
    ge = torch.full((4,), 1e7, device=DEV)
    got = mtp.mtp_token_logprobs_backward(logits, tokens, fw.lse, fw.entropy, ge, ge, 1e-3)
    assert torch.isfinite(got).all() and (got[:, ::2] == 0).all()


def test_calls_on_a_delayed_side_stream():
    """Calls with `stream`, late behind other work, while the current stream allocates and fills blocks of the sizes
    that they took: the same results as on the current stream."""
    g = gen(42)
    w = (randn(g, 640, 2048) * 0.02).to(BF16)
    x, logits = randn(g, 6, 2048).to(BF16), randn(g, 12, 5003)
    tokens, weights = torch.arange(12, dtype=torch.int32, device=DEV), randn(g, 12)
    cache, table = make_cache(g, [900, 60, 300], 2, 128, 32, "int8")
    lengths, q = ints([900, 60, 300]), randn(g, 3, 8, 128).to(BF16)

    def calls(**s):
        parts = mtp.mtp_q4_quantize(w, 32, True, **s)
        weight = mtp.Q4Weight(*parts, **s)
        del parts
        product = mtp.mtp_q4_matvec(mtp.Q4Weight.quantize(w, 64, **s), x, **s)
        scored = mtp.mtp_token_logprobs(logits, tokens, top=4, **s)
        grad = mtp.mtp_token_logprobs_backward(logits, tokens, scored.lse, scored.entropy, weights, **s)
        out, _ = mtp.mtp_kv_attention(cache, table, lengths, q, **s)
        return [weight.packed, product, out, grad, *scored]

    def sizes(t):
        return t.numel() * t.element_size()

    want = calls()
    taken = {640 * 1024, 640 * 64 * 2, 640 * 64, 640 * 32 * 2, 3 * 8 * 4, *map(sizes, want)}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = calls(stream=side)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in taken for _ in range(6)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all((t == 255).all() for t in junk)


def one_row(q, k, v, scale):
    q, k, v = q.cpu().double(), k.cpu().double(), v.cpu().double()
    if not k.shape[0]:
        z = torch.zeros_like(q)
        return z, z, torch.tensor(-math.inf).double(), torch.tensor(0.0)
    s = scale * (k @ q)
    ds = (q.shape[0] + 8) * U * abs(scale) * (k.abs() @ q.abs()).max() + 2.0 ** -21 * (1 + s.abs().max())
    p, chain = s.softmax(0), (64 + k.shape[0] / 16) * U
    o, size = p @ v, p @ v.abs()
    # weights have 11 bits, or 2^-32 of the largest
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * ds + 2 * chain) * size + k.shape[0] * 2.0 ** -32 * v.abs().amax(0) * p.max()
    lse = s.logsumexp(0)
    return o, tol, lse, ds + chain + 4 * U * lse.abs()


def tokens_of(cache, table_row, length, head):
    pages = table_row[:-(-length // cache.page_tokens)].long()
    out = []
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        x = ref.decode(codes[pages][:, head], cache.format) * scales[pages][:, head].cpu().double()[:, None, None]
        out.append(x.flatten(0, 1)[:length])
    return out


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("count", [1, 3])
@pytest.mark.parametrize("over,window", [(100, 200), (1, 7), (60, 70), (500, 40), (37, 0)])
def test_attention_longer_than_its_table_with_a_window(fmt, count, over, window):
    """What lies behind the table is left out, and nothing else: the window still counts from the true position."""
    g = gen(over)
    cap = 320
    cache, table = make_cache(g, [cap], 2, 64, 16, fmt)
    q = randn(g, count, 4, 64).to(BF16)
    out, lse = mtp.mtp_kv_attention(cache, table, ints([cap + over]), q, window=window)
    assert cache.read_errors() == mtp.MTP_DEVERR_PAGE
    for i in range(count):
        p = cap + over - count + i
        low = max(0, p - window + 1) if window else 0
        for h in range(4):
            k, v = tokens_of(cache, table[0], cap, h // 2)
            o, tol, l, ltol = one_row(q[i, h], k[low:p + 1], v[low:p + 1], 0.125)
            close(out[i, h], o, tol)
            close(lse[i, h], l, ltol)


@pytest.mark.parametrize("window", [0, 9])
def test_attention_keeps_the_places_of_tokens_within_the_bound(window):
    g = gen(31)
    lengths, counts = [50, 37], [6, 4]
    cache, table = make_cache(g, lengths, 1, 64, 16, "int8")
    q = randn(g, 10, 2, 64).to(BF16)
    full = mtp.mtp_kv_attention(cache, table, ints(lengths), q, starts=ints([0, 6, 10]), max_q=6, window=window)
    out, lse = torch.full_like(full[0], 9.0), torch.full_like(full[1], 9.0)
    mtp.mtp_kv_attention(cache, table, ints(lengths), q, starts=ints([0, 6, 10]), max_q=4, window=window, out=out, lse=lse)
    assert cache.read_errors() == mtp.MTP_DEVERR_OFFSETS
    for row in range(10):
        if row in (4, 5):
            assert (out[row] == 9).all() and (lse[row] == 9).all()
        else:
            for h in range(2):
                b, i = (0, row) if row < 6 else (1, row - 6)
                p = lengths[b] - counts[b] + i
                low = max(0, p - window + 1) if window else 0
                k, v = tokens_of(cache, table[b], lengths[b], 0)
                o, tol, l, ltol = one_row(q[row, h], k[low:p + 1], v[low:p + 1], 0.125)
                close(out[row, h], o, tol)
                close(lse[row, h], l, ltol)


def test_attention_bound_far_above_the_tokens():
    g = gen(34)
    cache, table = make_cache(g, [50, 37], 2, 64, 16, "int8")
    q = randn(g, 5, 4, 64).to(BF16)
    want = mtp.mtp_kv_attention(cache, table, ints([50, 37]), q, starts=ints([0, 2, 5]), max_q=5)
    got = mtp.mtp_kv_attention(cache, table, ints([50, 37]), q, starts=ints([0, 2, 5]), max_q=2 ** 31 - 1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_append_bound_far_above_the_tokens():
    g = gen(39)
    k, v = (randn(g, 40, 2, 64).to(BF16) for _ in range(2))
    caches = []
    for most in (37, 2 ** 31 - 1):
        cache = mtp.KvCache.allocate(6, 16, 2, 64, "e4m3")
        mtp.mtp_kv_append(cache, ints([[0, 1, 2], [3, 4, 5]]), ints([0, 7]), k, v, starts=ints([0, 37, 40]), max_new=most)
        assert cache.read_errors() == 0
        caches.append(cache)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(*(getattr(c, name) for c in caches))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("temperature", [1e20, 1e24, 2.0 ** 90, 1e28, 1e30, 1e33, 1e37])
def test_logprobs_at_very_high_temperatures(dtype, temperature):
    """Masked tokens have no probability where 1e30 / temperature is small, and logits at both ends of the type have one."""
    g = gen(37)
    for vocab in (50, 9000):
        logits = (randn(g, 7, vocab) * 3).to(dtype)
        logits[1, ::2] = -math.inf
        logits[2] = (randn(g, vocab) * 1e30).to(dtype)
        logits[2, 1::3] = -math.inf
        logits[3] = -math.inf
        logits[3, 4] = 1.0
        logits[4] = -math.inf
        logits[5] = torch.finfo(dtype).min
        logits[5, ::2] = torch.finfo(dtype).max
        logits[5, ::3] = -math.inf
        logits[6, 7] = math.nan
        tokens = ints([1, 2, 1, 4, 5, 7, 3])
        got = mtp.mtp_token_logprobs(logits, tokens, top=5, temperature=temperature)
        want = ref.logprobs(logits, tokens, temperature, 5)
        for name, (value, tol) in want.items():
            mine = getattr(got, name)
            if tol is None:
                assert torch.equal(mine[:6].cpu().long(), value[:6].long()), name
            else:
                close(mine[:6], value[:6], tol[:6], name)
                assert torch.isnan(mine[6]).all()
        gl, ge = randn(g, 7), randn(g, 7)
        grad = mtp.mtp_token_logprobs_backward(logits, tokens, got.lse, got.entropy, gl, ge, temperature)
        want, tol = exact_gradient(logits[:6], tokens[:6], temperature, gl[:6], ge[:6])
        # bf16: 2^-9 of a value (allowed: twice that), or half of the smallest subnormal
        close(grad[:6], want, tol + (2.0 ** -8 * want.abs() + 2.0 ** -134 if dtype == BF16 else 0.0) + 1e-44)


@pytest.mark.parametrize("temperature", [0.7, 0.3, 0.6, 1.0])
def test_rank_at_the_replacement_of_masked_logits(temperature):
    """A given logit near the number that stands in for -inf inside: the masked tokens do not come before it."""
    factor = torch.tensor(1.0 / temperature, dtype=F32)
    value = (torch.tensor(-1e30) / factor.clamp(min=1)).to(BF16)
    near = (value.view(torch.int16) + torch.tensor([-2, -1, 0, 1, 2], dtype=torch.int16)).view(BF16)
    for at in near:
        logits = torch.full((1, 20000), -math.inf, dtype=BF16, device=DEV)
        logits[0, 15000] = at
        logits[0, 3:9] = 1.0
        logits[0, 12000] = value.item() * 2
        got = mtp.mtp_token_logprobs(logits, ints([15000]), temperature=temperature)
        assert got.rank.item() == 6


@pytest.mark.parametrize("temperature", [4.4e-39, 6e-39, 1e-38])
def test_logprobs_at_the_lowest_temperatures(temperature):
    """One over the temperature is near fp32's end: the largest logit has all of the probability."""
    logits = torch.zeros(3, 5000, device=DEV)
    logits[0, 7] = 1e-3
    logits[1] = -1e-2
    logits[1, 9] = 0.5
    got = mtp.mtp_token_logprobs(logits, ints([7, 9, 3]), top=1, temperature=temperature)
    close(got.logprob, torch.tensor([0.0, 0.0, -math.log(5000)]), 2.0 ** -20)
    close(got.entropy, torch.tensor([0.0, 0.0, math.log(5000)]), 2.0 ** -18)
    assert got.rank.tolist() == [0, 0, 3] and got.top_ids[:, 0].tolist() == [7, 9, 0]


def one_dominant_token(g, fmt, dim, power):
    """A cache of 32 tokens whose first one alone has keys (the others' scores are 0, and their weights 2^power of its
    own) and no values, with the query and scale for it."""
    cache, table = make_cache(g, [32], 1, dim, 32, fmt)
    page = int(table[0, 0])
    cache.k_codes[page] = 0
    cache.k_codes[page, 0, 0, 0] = 64 if fmt == "int8" else 0x58   # 64, 16
    cache.v_codes[page, 0, 0] = 0
    cache.k_scales[page] = 1.0 / 64 if fmt == "int8" else 1.0 / 16
    q = torch.zeros(1, 1, dim, dtype=BF16, device=DEV)
    q[0, 0, 0] = 1.0
    return cache, table, q, float(torch.tensor(-power * math.log(2)))


def check_one_dominant_token(fmt, dim, power):
    cache, table, q, scale = one_dominant_token(gen(33), fmt, dim, power)
    out, lse = mtp.mtp_kv_attention(cache, table, ints([32]), q, scale=scale)
    k, v = tokens_of(cache, table[0], 32, 0)
    o, tol, l, ltol = one_row(q[0, 0], k, v, scale)
    close(out[0, 0], o, tol)
    close(lse[0, 0], l, ltol)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("power", [-12, -14, -18])
def test_attention_values_beside_a_large_weight_without_any(fmt, dim, power):
    check_one_dominant_token(fmt, dim, power)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("power", [-20.5, -24, -26])
def test_attention_small_weights_beside_a_large_one(fmt, dim, power):
    """What the others add is all of the output, however small their weights are."""
    check_one_dominant_token(fmt, dim, power)


_FROM_THREADS = """
import threading, torch, centroid_masked_sparse_gb300 as mtp
g = torch.Generator("cuda").manual_seed(1)
widths = [256, 16384, 512, 8192, 768, 12288, 1024, 4096]
for batch in (1, 9, 17, 25):
    for group in (32, 64, 128):
        weights, xs = [], []
        for cols in widths:
            w = (torch.randn(64, cols, device="cuda", generator=g) * 0.02).to(torch.bfloat16)
            weights.append(mtp.Q4Weight.quantize(w, group))
            xs.append(torch.randn(batch, cols, device="cuda", generator=g).to(torch.bfloat16))
        torch.cuda.synchronize()
        start, outs, errors = threading.Barrier(len(widths)), [None] * len(widths), []

        def call(i):
            try:
                start.wait()
                with torch.cuda.stream(torch.cuda.Stream()):
                    for _ in range(3):
                        outs[i] = mtp.mtp_q4_matvec(weights[i], xs[i])
            except Exception as e:
                errors.append(e)

        threads = [threading.Thread(target=call, args=(i,)) for i in range(len(widths))]
        [t.start() for t in threads], [t.join() for t in threads]
        torch.cuda.synchronize()
        assert not errors, errors
        for w, x, out in zip(weights, xs, outs):
            assert torch.equal(mtp.mtp_q4_matvec(w, x), out)
print("threads ok")
"""


def test_first_calls_from_several_threads():
    """Every thread's first call of a kernel needs another amount of shared memory; later ones of each size go through."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", _FROM_THREADS], cwd=root, capture_output=True, text=True, timeout=300)
    assert "threads ok" in run.stdout, run.stderr[-2000:]


def test_operators_from_several_threads():
    """Threads with a stream each, on one cache and one weight, get what a thread alone gets."""
    import threading
    g = gen(43)
    cache, table = make_cache(g, [9000, 60, 4000], 2, 128, 32, "int8")
    lengths, qs = ints([9000, 60, 4000]), [randn(g, 3, 8, 128).to(BF16) for _ in range(4)]
    weight = mtp.Q4Weight.quantize((randn(g, 5000, 1024) * 0.1).to(BF16))
    tokens = ints([3, 4, 5])

    def step(q):
        out, lse = mtp.mtp_kv_attention(cache, table, lengths, q)
        logits = mtp.mtp_q4_matvec(weight, out.flatten(1))
        scored = mtp.mtp_token_logprobs(logits, tokens, top=3)
        return [out, lse, logits, *scored, mtp.mtp_token_logprobs_backward(logits, tokens, scored.lse, scored.entropy, scored.logprob)]

    want = [step(q) for q in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got[i].append(step(qs[i]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(qs))]
    [t.start() for t in threads], [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(len(qs)):
        assert len(got[i]) == 10
        for results in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(results, want[i]))


def test_a_refused_device_leaves_no_error_behind():
    """Each call's status is its own: a call for a device that is not there, then calls that are right."""
    import ctypes
    from centroid_masked_sparse_gb300._lib import MtpQ4Desc, lib
    g = gen(44)
    w, x = (randn(g, 64, 256) * 0.1).to(BF16), randn(g, 3, 256).to(BF16)
    weight = mtp.Q4Weight.quantize(w)
    want, out = mtp.mtp_q4_matvec(weight, x), torch.empty(3, 64, device=DEV)
    desc = MtpQ4Desc.from_buffer_copy(weight.desc)
    desc.device = 99
    for call in (lambda: mtp.mtp_q4_quantize(w), lambda: mtp.Q4Weight.quantize(w), lambda: mtp.mtp_q4_matvec(weight, x)):
        assert lib().mtp_q4_matvec(ctypes.byref(desc), x.data_ptr(), 256, 3, out.data_ptr(), 0, 64, None) == -5
        call()
    assert torch.equal(mtp.mtp_q4_matvec(mtp.Q4Weight.quantize(w), x), want)


def test_workspace_of_a_device_that_is_not_there():
    import ctypes
    from centroid_masked_sparse_gb300._lib import MtpKvDesc, lib
    from centroid_masked_sparse_gb300.lm_ops import _batch_desc
    g = gen(35)
    cache, table = make_cache(g, [50], 2, 64, 16, "int8")
    seqs = _batch_desc(cache, table, ints([50]), None, 1, None)
    desc = MtpKvDesc.from_buffer_copy(cache.desc)
    desc.device = 99
    assert lib().mtp_kv_attention_workspace_bytes(ctypes.byref(desc), ctypes.byref(seqs), 4, 0, 0) == 0


@pytest.mark.parametrize("dim,batch,window", [(256, 1, 0), (128, 3, 0), (64, 1, 0), (256, 1, 12000)])
def test_attention_in_a_workspace_of_its_exact_size(dim, batch, window):
    """A split call: one byte less is refused; the size given is enough, nothing behind it is written, and its first part
    is zero again."""
    g = gen(dim + batch)
    lengths = [15000 - 700 * i for i in range(batch)]
    cache, table = make_cache(g, lengths, 1, dim, 32, "int8")
    q = randn(g, batch, 4, dim).to(BF16)
    want = mtp.mtp_kv_attention(cache, table, ints(lengths), q, window=window)
    need = mtp.mtp_kv_attention_workspace_bytes(cache, table, ints(lengths), batch, 4, window=window)
    assert need > mtp.MTP_KV_WORKSPACE_ZEROED and need % 4 == 0
    room = torch.full((need + 65536,), 0xa5, dtype=torch.uint8, device=DEV)
    room[:mtp.MTP_KV_WORKSPACE_ZEROED] = 0
    with pytest.raises(mtp.MtpError):
        mtp.mtp_kv_attention(cache, table, ints(lengths), q, window=window, workspace=room[:need - 1])
    for _ in range(3):
        got = mtp.mtp_kv_attention(cache, table, ints(lengths), q, window=window, workspace=room[:need])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (room[:mtp.MTP_KV_WORKSPACE_ZEROED] == 0).all() and (room[need:] == 0xa5).all()
    assert not (room[mtp.MTP_KV_WORKSPACE_ZEROED:need] == 0xa5).all()


def test_strides_of_one_token_or_head_do_not_matter():
    g = gen(36)
    cache, table = make_cache(g, [50], 1, 64, 16, "int8")
    wide = randn(g, 1, 68).to(BF16)
    q = wide[:, :64].unsqueeze(1)
    assert q.shape == (1, 1, 64) and q.stride(0) % 8
    want = mtp.mtp_kv_attention(cache, table, ints([50]), q.reshape(64).clone().view(1, 1, 64))
    got = mtp.mtp_kv_attention(cache, table, ints([50]), q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    new = [mtp.KvCache.allocate(4, 16, 1, 64, "int8") for _ in range(2)]
    for c, x in zip(new, (q, q.reshape(64).clone().view(1, 1, 64))):
        mtp.mtp_kv_append(c, ints([[0, 1]]), ints([3]), x, x)
    assert torch.equal(new[0].k_codes, new[1].k_codes) and torch.equal(new[0].v_scales, new[1].v_scales)


def test_q4_large_scales_and_small_inputs():
    """Scales and inputs whose products are of ordinary size although neither is."""
    g = gen(38)
    codes, scales, points = q4_weight(g, 64, 1024, 64, True)
    x = randn(g, 4, 1024).to(BF16)
    scales[3], scales[4] = 1e35, 1e30
    x[1] *= 2.0 ** -80
    x[2] *= 2.0 ** -110
    x[3] *= 2.0 ** 100
    want, tol = ref.q4_matvec(codes, scales, points, 64, x, 0.0, False)
    fits = want.abs() < 1e38
    fits[:, 3] = fits[:, 4] = False
    fits[1:3, 3] = fits[1:3, 4] = True
    close(mtp.mtp_q4_matvec(mtp.Q4Weight(codes, scales, points), x).cpu()[fits], want[fits], (tol + 1e-38)[fits])


def test_errors_of_calls_on_other_streams():
    """read_errors waits for every stream, and what it clears is cleared before later calls on any."""
    g = gen(45)
    cache, table = make_cache(g, [50], 1, 64, 16, "int8")
    q, bad, lengths, side = randn(g, 1, 2, 64).to(BF16), torch.full_like(table, -1), ints([50]), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            mtp.mtp_kv_attention(cache, bad, lengths, q)
        assert cache.read_errors() == mtp.MTP_DEVERR_PAGE
        mtp.mtp_kv_attention(cache, bad, lengths, q, stream=side)
        assert cache.read_errors() == mtp.MTP_DEVERR_PAGE
        assert cache.read_errors() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("share", [1, 3])
@pytest.mark.parametrize("length,window,bad", [(40, 0, "token 38"), (34, 0, "page 2"), (18, 2, "page 0"), (18, 2, "page 1"), (300, 0, "token 297"),
                                              (38, 3, "token 33")])
def test_attention_non_finite_values_that_a_query_does_not_see(fmt, dim, share, length, window, bad):
    """Five query tokens, some of which see a token with NaN codes or a page with a NaN or infinite scale: the others'
    outputs are what they would be without."""
    g = gen(length + dim)
    cache, table = make_cache(g, [length], 1, dim, 16, fmt)
    q = randn(g, 5, share, dim).to(BF16)
    scale = dim ** -0.5
    what, at = bad.split()
    at = int(at)
    if what == "token":
        if fmt == "int8":
            pytest.skip("int8 codes are all finite")
        cache.v_codes[int(table[0, at // 16]), 0, at % 16, ::3] = 0x7f
        cache.k_codes[int(table[0, at // 16]), 0, at % 16, 5] = 0xff
        spoilt = {at}
    else:
        cache.v_scales[int(table[0, at])] = math.nan if share == 1 else math.inf
        spoilt = set(range(at * 16, at * 16 + 16))
    out, lse = mtp.mtp_kv_attention(cache, table, ints([length]), q, window=window)
    seen_by_none = True
    for i in range(5):
        p = length - 5 + i
        low = max(0, p - window + 1) if window else 0
        if spoilt & set(range(low, p + 1)):
            assert not torch.isfinite(out[i]).all()
            continue
        seen_by_none = False
        for h in range(share):
            k, v = tokens_of(cache, table[0], length, 0)
            o, tol, l, ltol = one_row(q[i, h], k[low:p + 1], v[low:p + 1], scale)
            close(out[i, h], o, tol)
            close(lse[i, h], l, ltol)
    assert not seen_by_none


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,heads", [(64, 3), (128, 12), (256, 4)])
@pytest.mark.parametrize("lengths,counts,window", [
    ([20000], [1], 0), ([20000], [4], 0), ([9001, 15003], [3, 1], 0), ([20000], [1], 12345), ([18011, 300], [4, 2], 9000),
])
def test_attention_joined_from_several_clusters(fmt, dim, heads, lengths, counts, window):
    """Items of more than one cluster, whose sums go through global memory: each head size, with and without a window
    that spans several of them."""
    from tests.test_lm_ops_gpu import check_attention
    g = gen(sum(lengths) + dim)
    cache, table = make_cache(g, lengths, 1, dim, 64, fmt)
    q = randn(g, sum(counts), heads, dim).to(BF16)
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    need = mtp.mtp_kv_attention_workspace_bytes(cache, table, ints(lengths), sum(counts), heads, starts=ints(starts), max_q=max(counts),
                                                window=window)
    assert need > mtp.MTP_KV_WORKSPACE_ZEROED   # more than one cluster
    out, lse = check_attention(cache, table, lengths, counts, q, window=window)
    again = mtp.mtp_kv_attention(cache, table, ints(lengths), q, starts=ints(starts), max_q=max(counts), window=window)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dim,fmt", [(64, "int8"), (128, "e4m3"), (256, "int8")])
def test_attention_of_a_prompt(dim, fmt):
    """More query tokens than a tile holds rows, one prompt from its first token and one behind cached ones."""
    from tests.test_lm_ops_gpu import check_attention
    g = gen(dim)
    lengths, counts = [130, 300], [130, 77]
    cache, table = make_cache(g, lengths, 2, dim, 32, fmt)
    check_attention(cache, table, lengths, counts, randn(g, 207, 6, dim).to(BF16))
    check_attention(cache, table, lengths, counts, randn(g, 207, 6, dim).to(BF16), window=50)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_of_a_prompt_with_a_head_of_256(fmt):
    g = gen(46)
    befores, counts = [37, 0], [700, 1030]
    cache, table = make_cache(g, [b + n for b, n in zip(befores, counts)], 2, 256, 64, fmt)
    k, v = (randn(g, 1730, 2, 256).to(BF16) for _ in range(2))
    want = [ref.append(codes, scales, fmt, table, befores, [0, 700, 1730], x)
            for codes, scales, x in ((cache.k_codes, cache.k_scales, k), (cache.v_codes, cache.v_scales, v))]
    mtp.mtp_kv_append(cache, table, ints(befores), k, v, starts=ints([0, 700, 1730]), max_new=1030)
    for got, (codes, scales) in zip(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)), want):
        assert torch.equal(got[1].cpu(), scales) and torch.equal(got[0].cpu(), codes)


@pytest.mark.parametrize("rows,cols,batch", [(3000, 1024, 512), (257, 4096, 1024), (40000, 512, 200)])
def test_q4_of_a_prompt(rows, cols, batch):
    g = gen(rows)
    codes, scales, points = q4_weight(g, rows, cols, 64, True)
    x = randn(g, batch, cols).to(BF16)
    want, tol = ref.q4_matvec(codes, scales, points, 64, x, 0.0, True)
    close(mtp.mtp_q4_matvec(mtp.Q4Weight(codes, scales, points), x, out_dtype=BF16), want, tol)
