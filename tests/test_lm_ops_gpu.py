"""The operators around the head on the GPU, against plain 64-bit forms (lm_ops_reference): the sizes, masks,
strides and types where each can go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")

import centroid_masked_sparse_gb300 as mtp
from tests import lm_ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def close(got, want, tol, what=""):
    got, want, tol = got.detach().cpu().double(), want.double(), torch.as_tensor(tol).double().expand(want.shape)
    assert got.shape == want.shape, what
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN at other places"
    same = odd & ~torch.isnan(want)
    assert torch.equal(got[same], want[same]), f"{what}: infinities"
    off = (got - want).abs()[~odd] - tol[~odd]
    assert not off.numel() or off.max() <= 0, f"{what}: {int((off > 0).sum())} of {off.numel()} out, by {off.max():.3g}"


# ---------------------------------------------------------------------------
# 4-bit products
# ---------------------------------------------------------------------------
def q4_weight(g, rows, cols, group, zeros):
    codes = torch.randint(256, (rows, cols // 2), device=DEV, generator=g, dtype=torch.uint8)
    scales = (torch.rand(rows, cols // group, device=DEV, generator=g) * 0.02 + 1e-3).to(BF16)
    points = torch.randint(16, scales.shape, device=DEV, generator=g, dtype=torch.uint8) if zeros else None
    return codes, scales, points


@pytest.mark.parametrize("rows,cols,group,zeros,batch,softcap,dtype", [
    (1, 32, 32, False, 1, 0.0, F32),
    (1, 128, 128, True, 3, 0.0, BF16),
    (15, 64, 64, False, 8, 0.0, F32),
    (17, 96, 32, True, 9, 5.0, F32),
    (2048, 1536, 128, False, 1, 0.0, BF16),
    (513, 1536, 64, True, 2, 0.0, F32),
    (1000, 2592, 32, True, 23, 30.0, F32),
    (4099, 640, 128, False, 16, 0.0, F32),
    (333, 4096, 64, False, 32, 0.0, BF16),
    (40, 4096, 32, True, 33, 0.0, F32),
    (65, 16384, 64, True, 7, 0.0, F32),
    (129, 16384, 128, False, 64, 0.0, BF16),
    (31, 352, 32, False, 130, 0.0, F32),
    (70000, 256, 64, True, 5, 0.0, F32),
    (40000, 1056, 32, False, 17, 0.0, F32),
])
def test_q4_matvec(rows, cols, group, zeros, batch, softcap, dtype):
    g = gen(rows + cols)
    codes, scales, points = q4_weight(g, rows, cols, group, zeros)
    x = randn(g, batch, cols).to(BF16)
    got = mtp.mtp_q4_matvec(mtp.Q4Weight(codes, scales, points), x, out_dtype=dtype, softcap=softcap)
    want, tol = ref.q4_matvec(codes, scales, points, group, x, softcap, dtype == BF16)
    assert got.dtype == dtype
    close(got, want, tol)


# CTAs of 1 to 16 tiles (of 152), whose steps are shared among the warps, with x in one or several chunks
@pytest.mark.parametrize("rows, cols, group, zeros, batch", [
    (7000, 2048, 64, True, 8),
    (9000, 6656, 64, False, 1),
    (12000, 7936, 128, False, 13),
    (21488, 3392, 64, True, 5),
    (24320, 1024, 32, False, 16),
    (38912, 320, 64, True, 3),
    (20000, 4096, 32, False, 24),
    (31000, 2304, 64, True, 31),
])
def test_q4_steps_shared_among_warps(rows, cols, group, zeros, batch):
    g = gen(rows + batch)
    codes, scales, points = q4_weight(g, rows, cols, group, zeros)
    x = randn(g, batch, cols).to(BF16)
    w = mtp.Q4Weight(codes, scales, points)
    got = mtp.mtp_q4_matvec(w, x)
    want, tol = ref.q4_matvec(codes, scales, points, group, x, 0.0, False)
    close(got, want, tol)
    assert torch.equal(mtp.mtp_q4_matvec(w, x), got)


def test_q4_every_code_in_every_place():
    """Columns that each hold one code for one row: x is a unit vector, so each product is one exact weight."""
    g = gen(5)
    for group in (32, 64, 128):
        codes, scales, points = q4_weight(g, 48, 384, group, True)
        w = mtp.Q4Weight(codes, scales, points)
        want = ref.q4_weights(codes, scales, points, group).T
        for low in range(0, 384, 32):
            x = torch.zeros(32, 384, dtype=BF16, device=DEV)
            x[torch.arange(32), low + torch.arange(32)] = 1.0
            assert torch.equal(mtp.mtp_q4_matvec(w, x).cpu().double(), want[low:low + 32])


def test_q4_strides_and_padding():
    """Rows of codes, x and outputs further apart than their width; what lies between is neither read nor written."""
    g = gen(6)
    codes, scales, points = q4_weight(g, 100, 320, 64, True)
    wide = torch.full((100, 257), 255, dtype=torch.uint8, device=DEV)
    wide[:, :160] = codes
    x = torch.full((11, 512), math.nan, dtype=BF16, device=DEV)
    x[:, :320] = randn(g, 11, 320).to(BF16)
    out = torch.full((11, 131), 7.0, device=DEV)
    mtp.mtp_q4_matvec(mtp.Q4Weight(wide[:, :160], scales, points), x[:, :320], out=out[:, :100])
    want, tol = ref.q4_matvec(codes, scales, points, 64, x[:, :320], 0.0, False)
    close(out[:, :100], want, tol)
    assert (out[:, 100:] == 7).all()


def test_q4_extremes():
    """Zero and very small scales, large x; an infinity or NaN in x or a scale stays in its own row."""
    g = gen(7)
    codes, scales, _ = q4_weight(g, 64, 256, 64, False)
    scales[3] = 0.0
    scales[5] = 1e-30
    scales[6] = 1e30
    x = randn(g, 6, 256).to(BF16)
    x[1] *= 2.0 ** 60
    x[2] *= 2.0 ** -60
    w = mtp.Q4Weight(codes, scales)
    want, tol = ref.q4_matvec(codes, scales, None, 64, x, 0.0, False)
    fits = want.abs() < 1e38   # the others' partial sums leave fp32's range
    assert fits[1].sum() == 63 and fits.sum() == 6 * 64 - 1
    close(mtp.mtp_q4_matvec(w, x).cpu()[fits], want[fits], (tol + 1e-38)[fits])
    x[4, 7] = math.nan
    scales[9, 1] = math.nan
    got = mtp.mtp_q4_matvec(mtp.Q4Weight(codes, scales), x).cpu()
    assert torch.isnan(got[4]).all() and torch.isnan(got[:, 9]).all()
    keep = fits.clone()
    keep[4], keep[:, 9] = False, False
    close(got[keep], want[keep], (tol + 1e-38)[keep])


def test_q4_packed_layout():
    """The packed form, word by word as it is specified."""
    g = gen(10)
    for rows, cols, group in ((37, 352, 32), (16, 64, 64), (5, 640, 128)):
        codes, scales, points = (t.cpu() for t in q4_weight(g, rows, cols, group, True))
        packed = mtp.Q4Weight(*(t.to(DEV) for t in (codes, scales, points))).packed.cpu()
        tiles, blocks, steps, n = -(-rows // 16), -(-cols // 64), -(-cols // 256), 256 // group
        full = torch.zeros(tiles * 16, blocks * 32, dtype=torch.uint8)
        full[:rows, :cols // 2] = codes
        # [tile][half of 8 rows][g][block][half of 32 columns][t][4 bytes]
        want = full.view(tiles, 2, 8, blocks, 2, 4, 4).permute(0, 3, 2, 5, 4, 1, 6).reshape(-1)
        at = -(-want.numel() // 256) * 256
        assert torch.equal(packed[:want.numel()], want)
        for part in (scales.view(torch.uint8).view(rows, -1, 2), points[..., None]):
            full = torch.zeros(tiles * 16, steps * n, part.shape[-1], dtype=torch.uint8)
            full[:rows, :cols // group] = part
            want = full.view(tiles, 2, 8, steps, n, -1).permute(0, 3, 2, 4, 1, 5).reshape(-1)
            assert torch.equal(packed[at:at + want.numel()], want)
            at += -(-want.numel() // 256) * 256
        assert at == packed.numel()


def test_q4_rows_of_x_far_apart():
    """Each row of x has its own range: a large value beside small ones loses none of their bits down to 2^-25."""
    g = gen(26)
    codes, scales, points = q4_weight(g, 80, 512, 64, True)
    x = randn(g, 9, 512).to(BF16)
    x[:, 1::7] *= 2.0 ** -22
    x[3] *= 2.0 ** 100
    x[4] *= 2.0 ** -100
    x[5] = 0.0
    x[6] = 0.0
    x[6, 100] = 2.0 ** -130   # subnormal
    want, tol = ref.q4_matvec(codes, scales, points, 64, x, 0.0, False)
    close(mtp.mtp_q4_matvec(mtp.Q4Weight(codes, scales, points), x), want, tol + 2e-45)


def test_q4_beyond_32_bits():
    """Codes of over 4 GB: the last rows' offsets do not fit 32 bits."""
    rows, cols = 560_000, 16384
    codes = torch.zeros(rows, cols // 2, dtype=torch.uint8, device=DEV)
    scales = torch.ones(rows, cols // 128, dtype=BF16, device=DEV)
    g = gen(8)
    codes[-40:] = torch.randint(256, (40, cols // 2), device=DEV, generator=g, dtype=torch.uint8)
    x = randn(g, 1, cols).to(BF16)
    got = mtp.mtp_q4_matvec(mtp.Q4Weight(codes, scales), x)[:, -40:]
    want, tol = ref.q4_matvec(codes[-40:], scales[-40:], None, 128, x, 0.0, False)
    close(got, want, tol)


@pytest.mark.parametrize("rows,cols,group,zeros", [(1, 32, 32, False), (7, 128, 128, True), (300, 576, 64, True),
                                                   (64, 4096, 32, False)])
def test_q4_quantize(rows, cols, group, zeros):
    g = gen(9)
    wide = (randn(g, rows, cols + 8) * 0.02).to(BF16)
    w = wide[:, :cols]
    w[0, :group] = 0.0
    if rows > 2:
        w[2] = w[2].abs()   # no value below zero
    got = mtp.mtp_q4_quantize(w, group, zeros)
    codes, scales, points = ref.q4_quantize(w.contiguous(), group, zeros)
    assert torch.equal(got[1].cpu(), scales) and torch.equal(got[0].cpu(), codes)
    assert (got[2] is None) == (points is None)
    if zeros:
        assert torch.equal(got[2].cpu(), points)
    x = randn(g, 2, cols).to(BF16)
    want, tol = ref.q4_matvec(codes, scales, points, group, x, 0.0, False)
    close(mtp.mtp_q4_matvec(mtp.Q4Weight.quantize(w, group, zeros), x), want, tol)


# ---------------------------------------------------------------------------
# The 8-bit cache
# ---------------------------------------------------------------------------
def make_cache(g, lengths, kv_heads, dim, page, fmt, spread=1.0, extra=3):
    need = [-(-n // page) for n in lengths]
    total = sum(need) + extra
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    width = max(1, max(need))
    table = torch.full((len(lengths), width + 2), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    parts = []
    for _ in range(2):
        x = randn(g, total, kv_heads, page, dim)
        scales = x.abs().amax((2, 3)) / (127 if fmt == "int8" else 448)
        y = x / scales[..., None, None]
        codes = (y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)).view(torch.uint8)
        parts.append((codes, scales * spread ** (torch.rand(total, kv_heads, device=DEV, generator=g) * 2 - 1)))
    cache = mtp.KvCache(parts[0][0], parts[1][0], parts[0][1], parts[1][1], fmt)
    return cache, table[:, :width]


def starts_of(counts):
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    return starts


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def check_attention(cache, table, lengths, counts, q, window=0, scale=None, max_len=0, uniform=False):
    starts = starts_of(counts)
    out, lse = mtp.mtp_kv_attention(cache, table, ints(lengths), q, starts=None if uniform else ints(starts),
                                    max_q=None if uniform else max(counts), window=window, scale=scale, max_len=max_len)
    want = ref.attention(q, cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, cache.format, table, lengths,
                         starts, window, cache.head_dim ** -0.5 if scale is None else scale)
    close(out, want[0], want[1], "out")
    close(lse, want[2], want[3], "lse")
    assert cache.read_errors() == 0
    return out, lse


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,page,kv_heads,share", [(64, 16, 2, 1), (128, 32, 1, 4), (256, 64, 2, 2), (128, 48, 3, 5),
                                                     (256, 16, 1, 17), (64, 128, 4, 8)])
def test_attention_one_token(fmt, dim, page, kv_heads, share):
    lengths = [1, 2, 15, 16, 17, 0, page, page + 1, 3 * page - 1, 1000]
    g = gen(dim + page)
    cache, table = make_cache(g, lengths, kv_heads, dim, page, fmt)
    q = (randn(g, len(lengths), kv_heads * share, dim) * 1.5).to(BF16)
    check_attention(cache, table, lengths, [1] * len(lengths), q, uniform=True)


@pytest.mark.parametrize("window", [0, 1, 16, 37, 5000])
@pytest.mark.parametrize("dim,fmt", [(64, "e4m3"), (128, "int8"), (256, "e4m3")])
def test_attention_several_tokens(window, dim, fmt):
    """Ragged numbers of query tokens, a sequence without any, one whose queries begin before its first token."""
    lengths, counts = [40, 3, 700, 5, 129, 64], [5, 5, 8, 0, 1, 20]
    g = gen(window + dim)
    cache, table = make_cache(g, lengths, 2, dim, 32, fmt)
    q = randn(g, sum(counts), 6, dim).to(BF16)
    check_attention(cache, table, lengths, counts, q, window=window)


@pytest.mark.parametrize("max_len", [0, 1, 100, 20000])
@pytest.mark.parametrize("length", [1, 31, 4095, 20000])
def test_attention_long_rows_and_any_bound(length, max_len):
    """One sequence, split over the GPU; the bound on its length only decides the split."""
    g = gen(length)
    cache, table = make_cache(g, [length], 1, 128, 64, "int8")
    q = randn(g, 3, 8, 128).to(BF16)
    check_attention(cache, table, [length], [3], q, max_len=max_len, uniform=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attention_scales_far_apart(fmt):
    """Blocks whose scales differ by eight orders of magnitude, and blocks of zeros."""
    lengths = [500, 333]
    g = gen(11)
    cache, table = make_cache(g, lengths, 2, 128, 16, fmt, spread=1e4)
    cache.k_scales.clamp_(max=0.05)
    cache.v_scales[table[0, 3].item()] = 0.0
    cache.v_codes[table[0, 4].item()] = 0
    cache.k_codes[table[1, 2].item()] = 0
    cache.k_scales[table[1, 2].item()] = 0.0
    q = randn(g, 2, 4, 128).to(BF16)
    check_attention(cache, table, lengths, [1, 1], q, uniform=True)


@pytest.mark.parametrize("power", [-40, -12, 12, 40])
def test_attention_large_and_small_queries(power):
    """q far from 1 with the softmax scale that brings the scores back, and scores that single out one token."""
    g = gen(12)
    cache, table = make_cache(g, [300], 1, 64, 32, "int8")
    q = (randn(g, 1, 2, 64) * 2.0 ** power).to(BF16)
    check_attention(cache, table, [300], [1], q, scale=2.0 ** -power / 8, uniform=True)
    check_attention(cache, table, [300], [1], q, scale=2.0 ** -power * 3, uniform=True)


def test_attention_negative_and_zero_scale():
    g = gen(13)
    cache, table = make_cache(g, [77], 1, 64, 16, "e4m3")
    q = randn(g, 1, 2, 64).to(BF16)
    check_attention(cache, table, [77], [1], q, scale=-0.125, uniform=True)
    check_attention(cache, table, [77], [1], q, scale=0.0, uniform=True)


def test_attention_strides():
    """q as a slice of a fused projection: heads and tokens further apart than their width."""
    g = gen(14)
    lengths = [50, 90]
    cache, table = make_cache(g, lengths, 2, 64, 16, "int8")
    fused = randn(g, 2, 3, 9, 64).to(BF16)
    check_attention(cache, table, lengths, [1, 1], fused[:, 1, 2:6], uniform=True)
    check_attention(cache, table, lengths, [1, 1], fused[:, :, :4].transpose(1, 2)[:, :, 0], uniform=True)


def test_attention_ignores_what_it_must_not_see():
    """Codes behind the last token, pages of other sequences and unread table columns: NaN codes and bad ids."""
    g = gen(15)
    lengths, page = [21, 40], 16
    cache, table = make_cache(g, lengths, 1, 64, page, "e4m3")
    q = randn(g, 2, 2, 64).to(BF16)
    out, lse = check_attention(cache, table, lengths, [1, 1], q, uniform=True)
    nan = 0x7f
    used = set()
    for b, n in enumerate(lengths):
        for i in range(-(-n // page)):
            at = int(table[b, i])
            used.add(at)
            for codes in (cache.k_codes, cache.v_codes):
                codes[at, :, max(0, n - i * page):] = nan
    for at in set(range(cache.pages)) - used:
        cache.k_codes[at], cache.v_codes[at], cache.k_scales[at], cache.v_scales[at] = nan, nan, math.nan, math.nan
    again = mtp.mtp_kv_attention(cache, table, ints(lengths), q)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert cache.read_errors() == 0


def test_attention_window_reads_no_earlier_page():
    """Pages wholly before the window may have been given back: their ids are not read."""
    g = gen(16)
    lengths = [200]
    cache, table = make_cache(g, lengths, 1, 64, 16, "int8")
    q = randn(g, 1, 2, 64).to(BF16)
    want = mtp.mtp_kv_attention(cache, table, ints(lengths), q, window=40)
    table = table.clone()
    table[0, :10] = -1   # the window begins at 160
    got = mtp.mtp_kv_attention(cache, table, ints(lengths), q, window=40)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and cache.read_errors() == 0


def test_attention_flags_bad_pages_and_lengths():
    g = gen(17)
    lengths = [64, 64, 64]
    cache, table = make_cache(g, lengths, 1, 64, 16, "int8")
    q = randn(g, 3, 2, 64).to(BF16)
    good = table.clone()
    table = table.clone()
    table[0, 1], table[1, 2] = -5, cache.pages
    out, lse = mtp.mtp_kv_attention(cache, table, ints([64, 64, 10 ** 9]), q)
    assert cache.read_errors() == mtp.MTP_DEVERR_PAGE
    # the bad pages' tokens are left out: the same as attention over the other pages
    for b, gone in ((0, 1), (1, 2)):
        rest = torch.cat([good[b:b + 1, :gone], good[b:b + 1, gone + 1:]], 1).contiguous()
        want = ref.attention(q[b:b + 1], cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, "int8", rest, [48], [0, 1],
                             0, 0.125)
        close(out[b:b + 1], want[0], want[1])
        close(lse[b:b + 1], want[2], want[3])
    # bad starts: nothing outside the rows is touched
    out = torch.full((3, 2, 64), 9.0, dtype=BF16, device=DEV)
    mtp.mtp_kv_attention(cache, good, ints(lengths), q, starts=ints([0, 1, 9, 2]), max_q=2, out=out)
    assert cache.read_errors() == mtp.MTP_DEVERR_OFFSETS
    assert (out[1:] == 9).all() and not (out[0] == 9).any()


def test_attention_on_another_stream_and_repeated():
    """A side stream, with work behind it that makes the inputs late; the same call gives the same bits."""
    g = gen(18)
    lengths = [9000, 123, 4000]
    cache, table = make_cache(g, lengths, 2, 128, 32, "int8")
    q = randn(g, 3, 8, 128).to(BF16)
    want = check_attention(cache, table, lengths, [1] * 3, q, uniform=True)
    side = torch.cuda.Stream()
    late = torch.zeros_like(q)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
        out, lse = mtp.mtp_kv_attention(cache, table, ints(lengths), late)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for _ in range(5):
        got = mtp.mtp_kv_attention(cache, table, ints(lengths), q)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_captured_without_a_call_before():
    """Graphs own their workspaces: the second captured runs first, and eager calls that need more do not disturb them."""
    g = gen(22)
    lengths = [9000, 60, 4000]
    cache, table = make_cache(g, lengths, 2, 128, 32, "int8")
    q, lens = randn(g, 3, 8, 128).to(BF16), ints(lengths)
    want = check_attention(cache, table, lengths, [1] * 3, q, uniform=True)
    fresh = mtp.KvCache(cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, "int8")
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(mtp.mtp_kv_attention(fresh, table, lens, q))
        graphs.append(graph)
    many = randn(g, 24, 8, 128).to(BF16)
    mtp.mtp_kv_attention(fresh, table, lens, q)
    mtp.mtp_kv_attention(fresh, table, lens, many)
    for k in (1, 0, 1, 0):
        outs[k][0].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[k][0], want[0]) and torch.equal(outs[k][1], want[1])


def test_attention_on_two_streams_at_once():
    """Calls on two streams share nothing: each has its own workspace, and both give what a call alone gives."""
    g = gen(21)
    lengths = [9000, 60, 4000]
    cache, table = make_cache(g, lengths, 2, 128, 32, "int8")
    q = [randn(g, 3, 8, 128).to(BF16) for _ in range(2)]
    lens = ints(lengths)
    want = [mtp.mtp_kv_attention(cache, table, lens, x) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = ([], [])
    for _ in range(20):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(mtp.mtp_kv_attention(cache, table, lens, q[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_attention_in_a_graph():
    g = gen(19)
    cache, table = make_cache(g, [3000, 77], 1, 64, 16, "e4m3")
    lengths, q = ints([3000, 77]), randn(g, 2, 4, 64).to(BF16)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, lse = mtp.mtp_kv_attention(cache, table, lengths, q)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            mtp.mtp_kv_attention(cache, table, lengths, q, out=out, lse=lse)
    lengths.copy_(ints([2999, 5]))
    graph.replay()
    torch.cuda.synchronize()
    want = ref.attention(q, cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, "e4m3", table, [2999, 5], [0, 1, 2],
                         0, 0.125)
    close(out, want[0], want[1])
    close(lse, want[2], want[3])


def test_cache_beyond_32_bits():
    """A cache of over 4 GB of keys: the last pages' offsets do not fit 32 bits."""
    pages, heads, page, dim = 17000, 8, 128, 256
    cache = mtp.KvCache.allocate(pages, page, heads, dim, "int8")
    g = gen(20)
    n = 300
    table = ints([[pages - 1, 5, pages - 2]])
    k, v = (randn(g, n, heads, dim).to(BF16) for _ in range(2))
    mtp.mtp_kv_append(cache, table, ints([0]), k, v)
    q = randn(g, 1, heads, dim).to(BF16)
    ids = table[0].long()
    few = mtp.KvCache(cache.k_codes[ids], cache.v_codes[ids], cache.k_scales[ids], cache.v_scales[ids], "int8")
    for x, codes, scales in ((k, few.k_codes, few.k_scales), (v, few.v_codes, few.v_scales)):
        want = ref.append(torch.zeros_like(codes), torch.zeros_like(scales), "int8", ints([[0, 1, 2]]), [0], [0, n], x)
        assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])
    want = mtp.mtp_kv_attention(few, ints([[0, 1, 2]]), ints([n]), q)
    got = mtp.mtp_kv_attention(cache, table, ints([n]), q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,page,kv_heads,befores,counts", [
    (64, 16, 1, [0], [1]),
    (128, 16, 2, [0, 15, 16, 17, 31], [1, 1, 1, 1, 1]),
    (64, 32, 3, [5, 0, 31, 64, 100], [40, 1, 0, 33, 260]),
    (256, 64, 2, [63, 1], [2, 129]),
    (128, 1024, 1, [1000, 3], [30, 2000]),
    (64, 48, 2, [47, 48], [7, 96]),
])
def test_append(fmt, dim, page, kv_heads, befores, counts):
    g = gen(dim + page)
    ends = [b + n for b, n in zip(befores, counts)]
    cache, table = make_cache(g, ends, kv_heads, dim, page, fmt)
    starts = starts_of(counts)
    fused = randn(g, starts[-1], 2, kv_heads, dim).to(BF16)
    fused *= torch.rand(starts[-1], 1, 1, 1, device=DEV, generator=g) * 2   # some raise the scale, some do not
    if starts[-1] > 5:
        fused[3] = 0.0
    k, v = fused[:, 0], fused[:, 1]
    want = [ref.append(codes, scales, fmt, table, befores, starts, x)
            for codes, scales, x in ((cache.k_codes, cache.k_scales, k), (cache.v_codes, cache.v_scales, v))]
    mtp.mtp_kv_append(cache, table, ints(befores), k, v, starts=ints(starts), max_new=max(counts))
    for got, (codes, scales) in zip(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)), want):
        assert torch.equal(got[1].cpu(), scales)
        assert torch.equal(got[0].cpu(), codes)
    assert cache.read_errors() == 0


def test_append_zeros_and_non_finite():
    cache = mtp.KvCache.allocate(4, 16, 1, 64, "int8")
    table = ints([[2, 0]])
    zero = torch.zeros(1, 1, 64, dtype=BF16, device=DEV)
    cache.k_codes.fill_(3)
    mtp.mtp_kv_append(cache, table, ints([0]), zero, zero)
    assert float(cache.k_scales[2]) == 0 and (cache.k_codes[2, 0, 0] == 0).all() and (cache.k_codes[2, 0, 1:] == 3).all()
    odd = torch.ones(1, 1, 64, dtype=BF16, device=DEV)
    odd[0, 0, 3], odd[0, 0, 4], odd[0, 0, 5] = math.nan, math.inf, -math.inf
    mtp.mtp_kv_append(cache, table, ints([1]), odd, odd)
    codes = cache.k_codes[2, 0, 1].view(torch.int8)
    assert codes[3:6].tolist() == [0, 127, -127] and math.isfinite(float(cache.k_scales[2])) and (codes[6:] == 0).all()
    assert (cache.k_codes[2, 0, 0] == 0).all()


def test_append_flags_bad_pages_and_starts():
    cache = mtp.KvCache.allocate(3, 16, 1, 64, "int8")
    x = torch.ones(40, 1, 64, dtype=BF16, device=DEV)
    mtp.mtp_kv_append(cache, ints([[0, -1, 7]]), ints([0]), x, x)
    assert cache.read_errors() == mtp.MTP_DEVERR_PAGE
    assert (cache.k_codes[0] == 127).all() and (cache.k_codes[1:] == 0).all()
    mtp.mtp_kv_append(cache, ints([[1]]), ints([0]), x, x)   # 40 tokens, a table of one page
    assert cache.read_errors() == mtp.MTP_DEVERR_PAGE
    assert (cache.k_codes[1] == 127).all() and (cache.k_codes[2] == 0).all()
    mtp.mtp_kv_append(cache, ints([[2], [2]]), ints([0, -4]), x, x, starts=ints([0, 50, 4]), max_new=2)
    assert cache.read_errors() & mtp.MTP_DEVERR_OFFSETS
    assert (cache.k_codes[2] == 0).all()


def test_append_then_attend():
    """The cache as a model uses it: prompts, then tokens one by one, attended to after each."""
    g = gen(21)
    page, heads, dim, lengths = 16, 2, 64, [30, 7]
    cache = mtp.KvCache.allocate(12, page, heads, dim, "e4m3")
    table = ints([[0, 3, 6, 9], [1, 4, 7, 10]])
    starts = starts_of(lengths)
    k, v = (randn(g, starts[-1], heads, dim).to(BF16) for _ in range(2))
    mtp.mtp_kv_append(cache, table, ints([0, 0]), k, v, starts=ints(starts), max_new=30)
    for step in range(4):
        k, v = ((randn(g, 2, heads, dim) * (1 + step)).to(BF16) for _ in range(2))
        mtp.mtp_kv_append(cache, table, ints([n + step for n in lengths]), k, v)
        q = randn(g, 2, 4, dim).to(BF16)
        check_attention(cache, table, [n + step + 1 for n in lengths], [1, 1], q, uniform=True)


# ---------------------------------------------------------------------------
# Token log probabilities
# ---------------------------------------------------------------------------
def check_logprobs(logits, tokens, temperature=1.0, top=0):
    got = mtp.mtp_token_logprobs(logits, tokens, top=top, temperature=temperature)
    want = ref.logprobs(logits, tokens, temperature, top)
    for name, (value, tol) in want.items():
        mine = getattr(got, name)
        if tol is None:
            assert torch.equal(mine.cpu().long(), value.long()), name
        else:
            close(mine, value, tol, name)
    return got


def rows_of(g, rows, vocab, dtype, spread=2.5):
    logits = (randn(g, rows, vocab) * spread).to(dtype)
    tokens = torch.randint(vocab, (rows,), device=DEV, generator=g).to(torch.int32)
    return logits, tokens


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,top,temperature", [
    (1, 1, 1, 1.0), (1, 2, 5, 1.0), (3, 31, 32, 0.5), (2, 33, 3, 1.0), (5, 255, 0, 2.0), (4, 4097, 20, 0.75), (2, 5000, 32, 1.0),
    (1, 262144, 20, 1.0), (7, 50021, 5, 0.25), (300, 1000, 8, 1.0), (40, 32003, 1, 1.5), (1, 100003, 32, 1.0),
    (700, 3001, 32, 1.0),
])
def test_logprobs(dtype, rows, vocab, top, temperature):
    logits, tokens = rows_of(gen(rows + vocab), rows, vocab, dtype)
    if rows > 1:
        tokens[1] = -1
    if rows > 2:
        tokens[2] = vocab
    check_logprobs(logits, tokens, temperature, top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [40, 5003, 262144])
def test_logprobs_masked_rows(dtype, vocab):
    """-inf masks that leave most, few, one or no token; a given token under the mask; the type's lowest value."""
    g = gen(vocab)
    logits, tokens = rows_of(g, 8, vocab, dtype)
    keep = torch.rand(8, vocab, device=DEV, generator=g) < torch.tensor([0.9, 0.5, 0.1, 10 / vocab, 0, 0, 0.5, 0.5], device=DEV)[:, None]
    keep[5, vocab // 2] = True
    logits.masked_fill_(~keep, -math.inf)
    tokens[6] = int((~keep[6]).nonzero()[0])
    lowest = torch.finfo(dtype).min
    logits[7].masked_fill_(~keep[7], lowest)
    check_logprobs(logits, tokens, top=20)
    logits[0], logits[1] = lowest, lowest
    logits[1, vocab - 1] = 0
    check_logprobs(logits, tokens, top=32)


@pytest.mark.parametrize("order", ["rising", "falling", "equal", "two values", "late peaks", "one per 16"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [1000, 70001])
def test_logprobs_orders_and_ties(order, dtype, vocab):
    """Orders that keep beating what was found so far, and ties, which go to the lower id."""
    at = torch.arange(vocab, device=DEV)
    x = {"rising": at / vocab * 20, "falling": -(at / vocab) * 20, "equal": torch.full((vocab,), 1.5, device=DEV),
         "two values": (at % 7 == 3).float(), "late peaks": (at > vocab - 50).float() * at / vocab * 9,
         "one per 16": (at % 16 == 5).float() * (3 + at / vocab)}[order]
    logits = x.to(dtype).repeat(3, 1)
    logits[2] = logits[2].flip(0)
    check_logprobs(logits, ints([0, vocab - 1, vocab // 2]), top=32)


def test_logprobs_zero_signs_and_large_values():
    logits = torch.zeros(3, 500, device=DEV)
    logits[0, ::2] = -0.0
    logits[1] = torch.linspace(-1e4, 1e4, 500, device=DEV)
    logits[2] = 1e30
    check_logprobs(logits, ints([1, 499, 77]), top=8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_logprobs_non_finite(dtype, bad):
    """A NaN or +inf spoils its own row and no other."""
    logits, tokens = rows_of(gen(3), 3, 9001, dtype)
    want = mtp.mtp_token_logprobs(logits, tokens, top=4)
    for at in (0, 4500, 9000):
        spoilt = logits.clone()
        spoilt[1, at] = bad
        got = mtp.mtp_token_logprobs(spoilt, tokens, top=4)
        for name in ("logprob", "entropy", "lse", "top_logprobs"):
            assert torch.isnan(getattr(got, name)[1]).all(), name
        for name in got._fields:
            a, b = getattr(got, name), getattr(want, name)
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset,extra", [(0, 1), (1, 0), (3, 5), (7, 1)])
def test_logprobs_strides_and_alignment(dtype, offset, extra):
    g = gen(offset)
    wide = torch.full((6, 3000 + 16), math.inf, device=DEV, dtype=dtype)
    logits = wide[:, offset:offset + 2999 + extra]
    logits.copy_(randn(g, *logits.shape))
    tokens = torch.randint(2999, (6,), device=DEV, generator=g).to(torch.int32)
    got = check_logprobs(logits, tokens, top=6)
    gl, ge = randn(g, 6), randn(g, 6)
    out = torch.full_like(wide, 5.0)
    view = out[:, 2:2 + logits.shape[1]]
    mtp.mtp_token_logprobs_backward(logits, tokens, got.lse, got.entropy, gl, ge, out=view)
    want, tol = ref.logprobs_grad(logits, tokens, 1.0, gl, ge, dtype == BF16)
    close(view, want, tol)
    assert (out[:, :2] == 5).all() and (out[:, 2 + logits.shape[1]:] == 5).all()


def test_logprobs_partial_outputs():
    """Outputs that a caller leaves out, and reuse of an earlier result."""
    logits, tokens = rows_of(gen(4), 5, 2000, F32)
    full = mtp.mtp_token_logprobs(logits, tokens, top=3)
    again = mtp.TokenLogprobs(*(torch.zeros_like(t) for t in full))
    assert mtp.mtp_token_logprobs(logits, tokens, top=3, out=again) is again
    some = mtp.TokenLogprobs(None, torch.zeros(5, device=DEV), None, torch.zeros(5, device=DEV), None, None)
    mtp.mtp_token_logprobs(logits, None, out=some)
    for a, b in zip(full, again):
        assert torch.equal(a, b)
    assert torch.equal(some.entropy, full.entropy) and torch.equal(some.lse, full.lse)


def test_logprobs_beyond_32_bits():
    rows, vocab = 8200, 262144
    logits = torch.zeros(rows, vocab, dtype=BF16, device=DEV)
    g = gen(22)
    logits[-2:] = randn(g, 2, vocab).to(BF16)
    tokens = torch.full((rows,), 17, dtype=torch.int32, device=DEV)
    got = mtp.mtp_token_logprobs(logits, tokens, top=3)
    want = ref.logprobs(logits[-2:], tokens[-2:], 1.0, 3)
    for name, (value, tol) in want.items():
        mine = getattr(got, name)[-2:]
        assert torch.equal(mine.cpu().long(), value.long()) if tol is None else close(mine, value, tol, name) is None
    gl = torch.ones(rows, device=DEV)
    grad = mtp.mtp_token_logprobs_backward(logits, tokens, got.lse, got.entropy, gl, out=logits.clone())
    want, tol = ref.logprobs_grad(logits[-2:], tokens[-2:], 1.0, gl[-2:], None, True)
    close(grad[-2:], want, tol)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,temperature,entropy", [(1, 1, 1.0, True), (3, 7, 0.5, True), (2, 4096, 1.0, False),
                                                            (5, 5003, 1.5, True), (33, 32003, 1.0, True),
                                                            (1, 262144, 0.75, False)])
def test_gradient(dtype, rows, vocab, temperature, entropy):
    g = gen(rows + vocab)
    logits, tokens = rows_of(g, rows, vocab, dtype)
    if rows > 2:
        tokens[1] = -1
        logits[2, ::3] = -math.inf
        tokens[2] = 1
    if rows > 4:
        logits[4] = -math.inf
    fw = mtp.mtp_token_logprobs(logits, tokens, temperature=temperature)
    gl, ge = randn(g, rows), randn(g, rows) if entropy else None
    got = mtp.mtp_token_logprobs_backward(logits, tokens, fw.lse, fw.entropy, gl, ge, temperature)
    want, tol = ref.logprobs_grad(logits, tokens, temperature, gl, ge, dtype == BF16)
    close(got, want, tol)
    if entropy:   # the entropy's alone, and in place
        only = logits.clone()
        mtp.mtp_token_logprobs_backward(only, None, fw.lse, fw.entropy, None, ge, temperature, out=only)
        want, tol = ref.logprobs_grad(logits, tokens, temperature, None, ge, dtype == BF16)
        close(only, want, tol)


def test_gradient_against_differences():
    """Central differences of the forward call itself, through autograd's entry: their error is the third
    derivative's h^2 / 6 (at most 0.1 for ln p, 2 for the entropy, of logits near 1) and twice the values' own
    error (2^-22 of about 16) over 2 h."""
    g = gen(23)
    logits, tokens = rows_of(g, 3, 37, F32, spread=1.0)
    wl, we = randn(g, 3), randn(g, 3)
    leaf = logits.clone().requires_grad_()
    logprob, entropy = mtp.token_logprobs(leaf, tokens, 0.8)
    (logprob * wl + entropy * we).sum().backward()
    h = 2.0 ** -6
    for i in range(37):
        values = []
        for sign in (h, -h):
            moved = logits.clone()
            moved[:, i] += sign
            got = mtp.mtp_token_logprobs(moved, tokens, temperature=0.8)
            values.append((got.logprob * wl + got.entropy * we).double())
        differences = (values[0] - values[1]) / (2 * h)
        weight = wl.abs() + we.abs()
        tol = (weight * (2 * h * h / 6 * 2 + 2 * 2.0 ** -22 * 16 / (2 * h))).cpu().double()
        close(leaf.grad[:, i], differences.cpu(), tol)


def test_autograd_through_a_linear_head():
    """token_logprobs as the loss of a linear head in bf16: the gradients of its weight and input."""
    g = gen(24)
    h = randn(g, 9, 64).to(BF16).requires_grad_()
    w = (randn(g, 500, 64) * 0.2).to(BF16).requires_grad_()
    tokens = torch.randint(500, (9,), device=DEV, generator=g).to(torch.int32)
    logits = h @ w.T
    logits.retain_grad()
    loss = -mtp.token_logprobs(logits, tokens)[0].mean()
    loss.backward()
    want, tol = ref.logprobs_grad(logits.detach(), tokens, 1.0, torch.full((9,), -1 / 9), None, True)
    close(logits.grad, want, tol)
    assert torch.equal(w.grad, logits.grad.T @ h) and torch.equal(h.grad, logits.grad @ w)
