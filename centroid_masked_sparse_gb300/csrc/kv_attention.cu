// Attention of one or a few query tokens per sequence over the paged 8-bit cache.
//
// Mathematics.  For a query row (a query token and a head), s_j = scale * k_scale * (q . c_j)
// over key codes c_j, p_j = 2^(s_j - m) in units of log2, o = sum p_j v_scale v_j / sum p_j.
// Both products run on the tensor cores (mma m16n8k16, fp16 in, fp32 sums) with the codes as
// the 16-row operand: S^T = K Q^T, 16 tokens by 8 query rows, and O^T = V^T P^T, 16 columns
// of the head by 8 query rows, so the heads that share a kv head and a call's query tokens
// fill the 8 columns.  Codes become fp16 as follows:
//  - int8 keys: the byte c + 128, masked in place, is the fp16 subnormal (c + 128) * 2^-24; the
//    128 * sum q leaves the sum through its start, in fp32;
//  - int8 values: 1152 + c, less 1152, exact.  (In the keys' way the sums would carry 128 beside
//    each code, and a token of large weight and small values would cost the others their bits.)
//  - e4m3: cvt to fp16, exact.
// q, which has 8 significant bits, is fp16 times a power of two per row; p is rounded to
// fp16's 11 bits, and the same rounded p make the denominator.  The sums of a block of 16
// tokens start at zero and are added, times v_scale, to the row's in fp32: blocks have their
// own scales.  m is 7 below the row's maximum so far, or up to 15: p stays within 2^15, most
// blocks need no maximum across lanes, and weights down to 2^-21 of the largest keep their 11
// bits (those below are fp16 subnormals, off by up to 2^-32 of the largest).
//
// Split.  A warp reads blocks of 16 tokens, two steps ahead, each lane the
// pieces of its own operands (cp.async into its own slots: no barrier).  The CTAs of an item
// (a sequence, a kv head, a tile of query rows) share its blocks; eight of them form a
// cluster and join their sums through distributed shared memory, each one slice of the
// head's columns.  Only an item with more than one cluster goes through global memory: the
// last cluster to arrive, per slice, adds the others' sums in their order.
//
// What bounds it: latency, and the ends of unequal CTAs.  64 ragged sequences of up to 8191
// tokens (8 kv heads of 128, 617 MB) take 127.6 us, 4.8 TB/s, with instructions in 0.46 of the
// issue slots and the tensor pipe 13 % busy: every item gets the same number of CTAs, whatever
// its length.  One sequence of 65519 tokens (one kv head of 256, 33.6 MB) takes 16.4 us: its
// chain of look-ups, few steps and joins.  16 sequences of up to five query tokens in a window
// of 512 take 12.6 us, one pass through that chain.  A warp per query row on the CUDA cores took
// 20.8 ms, 3 ms and 138 us.
#include <algorithm>

#include "lm_ops.h"

namespace mtp {

namespace {

constexpr int kW = 4;            // warps of a CTA
template <int D> constexpr int kStageOf = D == 256 ? 8192 : 4096;   // bytes of codes of a step
// Blocks of 16 tokens that a CTA should have at least (65519 tokens, D = 256: 17.2 us, with eight
// 25.6, with 24 20.9; 16 sequences of 8 tokens, a window of 1024 and 8 kv heads of 128: 34.6, 34.6
// and 31.8).
constexpr int kMinBlocks = 16;
constexpr int kMaxCluster = 8;
constexpr int kMaxSplits = 512;
constexpr float kHeadroom = 7.f;   // the weights' exponents above their reference
// A cluster's sums of R rows in global memory, and their statistics once for each slice.
constexpr int partial_floats(int D, int R) { return R * D + kMaxCluster * R * 4; }

template <bool INT8> __device__ __forceinline__ void key_operands(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if (INT8) {   // bytes (0, 2) and (1, 3)
        lo = (w & 0x00ff00ffu) ^ 0x00800080u;
        hi = (w >> 8 & 0x00ff00ffu) ^ 0x00800080u;
    } else {      // bytes (0, 1) and (2, 3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)w));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
    }
}

// Bytes 0..3 of two tokens' words: pairs (a_i, b_i).
template <bool INT8> __device__ __forceinline__ void value_operands(uint32_t a, uint32_t b, uint32_t (&v)[4])
{
    const uint32_t x = __byte_perm(a, b, INT8 ? 0x5410 : 0x5140), y = __byte_perm(a, b, INT8 ? 0x7632 : 0x7362);
    if (INT8) {
        auto code = [](uint32_t w) {   // 1152 + c, less 1152
            uint32_t r;
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"((w & 0x00ff00ffu) ^ 0x64806480u), "r"(0x64806480u));
            return r;
        };
        v[0] = code(x), v[1] = code(x >> 8), v[2] = code(y), v[3] = code(y >> 8);
    } else {
        key_operands<INT8>(x, v[0], v[1]);
        key_operands<INT8>(y, v[2], v[3]);
    }
}

// Four CTAs per SM (64 ragged sequences, D = 128, with the zeroing of a graph's workspace: 128.8
// us, with three and steps of eight kilobytes 137.9) where their sums leave the registers for it.
constexpr int ctas_per_sm(int D, int NT) { return NT > 1 ? 2 : D > 128 ? 3 : 4; }
// The rings of a CTA's warps, or the sums that take their place.
constexpr int ring_bytes(int D, int NT)
{
    const int ring = kW * 2 * (D == 256 ? kStageOf<256> : kStageOf<64>), sums = kW * NT * 8 * D * 4;
    return ring > sums ? ring : sums;
}


// Of a block that not every row sees whole: where a row does not see a token its weight is 0, but
// 0 times a NaN or an infinity is not.  NaN codes become 0, and the columns that they (or all, that
// a scale which is not finite) spoil are noted for those of the lane's rows that see the token; they
// end as NaN.  Returns whether there are any.  A call, and with the number of the warp as a value
// that the compiler knows to be uniform, since the loop takes it badly inside: 16 sequences of 4
// query tokens in e4m3 62.0 us, inlined 66.0, without all of this 62.4.
template <int D, bool INT8, int NT>
__device__ __noinline__ bool note_spoilt(uint8_t *values, float scale, uint32_t *spoilt, int pos, long long base, int r0, int share,
                                         int live, int lo, int end, int window)
{
    constexpr int E = D < 128 ? D / 8 : 16, PIECES = D < 128 ? 1 : D / 128, WORDS = E / 4;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    auto word = [&](int i, int j, int k) {   // word k of the lane's token i, piece j
        return (uint32_t *)(values + (D < 128 ? i / 2 * 512 + i % 2 * 8 : (j * 4 + i) * 512)) + k;
    };
    auto nans = [](uint32_t w) { return INT8 ? 0u : __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); };
    const bool all = !(fabsf(scale) < INFINITY);
    uint32_t some = all;
    if (!INT8) {
#pragma unroll 1
        for (int i = 0; i < 4 * PIECES; ++i)
#pragma unroll
            for (int k = 0; k < WORDS; ++k) some |= nans(*word(i % 4, i / 4, k));
    }
    if (!__any_sync(~0u, some != 0)) return false;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        uint32_t columns = all ? ~0u : 0u;   // of the token, one bit each
#pragma unroll 1
        for (int k = 0; k < (INT8 ? 0 : PIECES * WORDS); ++k) {
            uint32_t *w = word(i, k / WORDS, k % WORDS);
            const uint32_t bad = nans(*w);
            *w &= ~bad;
            columns |= ((bad & 0x08040201u) * 0x01010101u >> 24) << (k * 4);
        }
#pragma unroll 1
        for (int other = 0; other < 4; ++other) {   // the lanes with the other tokens of these columns
            const uint32_t theirs = __shfl_sync(~0u, columns, g * 4 + other);
            const int token = pos + 2 * other + i % 2 + i / 2 * 8;
#pragma unroll 1
            for (int r = 0; r < NT * 2; ++r) {
                const long long at = base + (r0 + min(r / 2 * 8 + 2 * t + r % 2, live - 1)) / share;
                if (token >= lo && token < end && token <= at && !(window > 0 && at - token >= window)) spoilt[r * kW * 32] |= theirs;
            }
        }
    }
    return true;
}

// D: columns of a head; NT: query rows / 8.
template <int D, bool INT8, int NT>
__global__ void __launch_bounds__(kW * 32, ctas_per_sm(D, NT)) k_kv_attention(KvAttentionParams p)
{
    constexpr int kStage = kStageOf<D>;
    constexpr int U = kStage / (32 * D);       // blocks of 16 tokens in a step
    constexpr int J = D / 64;                  // pieces of 64 columns of a key
    constexpr int MT = D / 16;                 // tiles of 16 columns of a value
    constexpr int E = D < 128 ? D / 8 : 16;    // columns of a lane in a piece of 128 (64)
    constexpr int R = NT * 8;
    constexpr float UNIT = INT8 ? 16777216.f : 1.f;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_factor[R], s_bias[R];
    __shared__ float s_stat[kW][3][R];         // maximum, sum of rounded p, sum of p of each warp
    __shared__ __align__(16) float4 s_total[R];   // the same of the CTA, read by the cluster
    __shared__ uint32_t s_last;
    __shared__ uint32_t s_spoilt[NT * 2][kW * 32];   // a lane's columns that values spoil, of each of its rows
    const KvParams &c = p.c;
    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int share = p.heads / c.kv_heads;

    // the item and its rows; everything that ends the kernel early holds for the whole cluster
    const int split = blockIdx.x, b = blockIdx.z, h = blockIdx.y / p.row_tiles;
    const long long item = (long long)b * gridDim.y + blockIdx.y;
    wait_for_previous();
    const long long length = __ldg(c.lengths + b);
    int row0, n;
    const int brought = kv_rows(c, b, &row0, &n);
    const int r0 = (blockIdx.y - h * p.row_tiles) * R, live = min(R, n * share - r0);
    if (live <= 0) return;
    const int cap = c.table_width * c.page_tokens;
    if ((length < 0 || length > cap) && c.err && threadIdx.x == 0) atomicOr(c.err, MTP_DEVERR_PAGE);
    // query i stands at position base + i; positions [lo, end) are seen by some row
    const long long base = length - brought;
    const int q_lo = r0 / share, q_hi = (r0 + live - 1) / share;
    const int lo = p.window > 0 ? (int)max(0ll, base + q_lo - p.window + 1) : 0;
    const int end = (int)max(0ll, min(base + q_hi + 1, (long long)cap));
    const int b_lo = lo / 16, blocks = end > lo ? (end + 15) / 16 - b_lo : 0;
    const int csize = (int)cluster_size(), crank = (int)cluster_rank();
    const int used = min(p.splits, max(1, (blocks + kMinBlocks - 1) / kMinBlocks));
    const int clusters = (used + csize - 1) / csize, ck = split / csize;
    if (ck >= clusters) return;
    const int parts = clusters * csize, per = blocks / parts, rest = blocks - per * parts;
    const int s_lo = b_lo + per * split + min(split, rest), s_hi = s_lo + per + (split < rest);

    // this warp's rows of queries, on their way while the first pages are looked up
    constexpr int QR = R / kW;
    uint4 q_in[QR];
#pragma unroll
    for (int i = 0; i < QR; ++i) {
        const int row = r0 + warp + i * kW;
        q_in[i] = make_uint4(0, 0, 0, 0);
        if (warp + i * kW < live && lane < D / 8)
            q_in[i] = ld_ro16(p.q + (long long)(row0 + row / share) * p.q_token + (long long)(h * share + row % share) * p.q_head + lane * 8);
    }

    // loads: a lane copies what it will read.  Keys: pieces (j, row half), 16 bytes of token
    // g (+ 8); values: of tokens 2t, 2t + 1, 2t + 8, 2t + 9, the columns of g.
    uint8_t *ring = smem + warp * 2 * kStage + lane * 16;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    const int page_blocks = c.page_tokens / 16;
    const int32_t *table = c.table + b * c.ld_table;
    // of the step at hand, the next one, and the page and the block in it of the one after
    float ks[U], vs[U], n_ks[U], n_vs[U];
    bool ok[U], n_ok[U];
    struct Place {
        int page, block;
    };
    Place n_place[U];
    auto fetch = [&](int it, Place (&to)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int block = s_lo + (it * kW + warp) * U + u;
            const int column = p.page_magic ? (int)__umulhi(block, p.page_magic) : block;   // block / page_blocks
            to[u].page = block < s_hi ? __ldg(table + column) : -1;
            to[u].block = block - column * page_blocks;
        }
    };
    auto load = [&](int it, const Place (&from)[U], float (&ks)[U], float (&vs)[U], bool (&ok)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int block = s_lo + (it * kW + warp) * U + u, page = from[u].page;
            ok[u] = page >= 0 && page < c.pages;
            if (!ok[u]) {
                if (block < s_hi && c.err && lane == 0) atomicOr(c.err, MTP_DEVERR_PAGE);
                continue;
            }
            const long long ph = (long long)page * c.kv_heads + h;
            const long long at = (ph * c.page_tokens + from[u].block * 16) * D;
            ks[u] = __ldg(c.k_scales + ph);
            vs[u] = __ldg(c.v_scales + ph);
            const int pos = block * 16;
            const bool whole = pos >= lo && pos + 16 <= end;
            // tokens outside [lo, end) are not read: zeros take their place
            auto bytes = [&](int token) { return whole || (pos + token >= lo && pos + token < end) ? 16 : 0; };
            uint32_t dst = ring_s + (it & 1) * kStage + u * 32 * D;
            const uint8_t *k = c.k_codes + at + g * D + t * 16;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int size = bytes(g + half * 8);
#pragma unroll
                for (int j = 0; j < J; ++j) cp_async16_part(dst + (j * 2 + half) * 512, k + half * 8 * D + j * 64, size);
            }
            dst += 16 * D;
            const uint8_t *v = c.v_codes + at + 2 * t * D + g * E;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int off = i % 2 + i / 2 * 8, size = bytes(2 * t + off);
                if (D < 128) {
                    cp_async8_part(dst + i / 2 * 512 + i % 2 * 8, v + off * D, size / 2);
                } else {
#pragma unroll
                    for (int j = 0; j < D / 128; ++j) cp_async16_part(dst + (j * 4 + i) * 512, v + off * D + j * 128, size);
                }
            }
        }
    };
    auto advance = [&] {
#pragma unroll
        for (int u = 0; u < U; ++u) ks[u] = n_ks[u], vs[u] = n_vs[u], ok[u] = n_ok[u];
    };
    {
        Place first[U], second[U];
        fetch(0, first);
        fetch(1, second);
        fetch(2, n_place);
        load(0, first, ks, vs, ok);
        cp_async_commit();
        load(1, second, n_ks, n_vs, n_ok);
        cp_async_commit();
    }

    // each row's power of two, and the row in the operand's order
    uint4 *s_q = (uint4 *)(smem + ring_bytes(D, NT));   // [piece of 64][half of a lane's 16][NT][lane]
#pragma unroll
    for (int i = 0; i < QR; ++i) {
        const int r = warp + i * kW;
        const uint4 v = q_in[i];
        uint32_t top = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        top = __reduce_max_sync(~0u, max(top >> 16, top & 0xffffu));
        const uint32_t e = fp16_factor_field(top);
        const float f = __uint_as_float(e << 23);
        const float x0 = bf_lo(v.x) * f, x1 = bf_hi(v.x) * f, x2 = bf_lo(v.y) * f, x3 = bf_hi(v.y) * f;
        const float x4 = bf_lo(v.z) * f, x5 = bf_hi(v.z) * f, x6 = bf_lo(v.w) * f, x7 = bf_hi(v.w) * f;
        if (lane < D / 8)   // columns 8 * lane of the row: piece lane / 8, lane (r % 8, lane % 8 / 2)
            s_q[((lane / 8 * 2 + lane % 2) * NT + r / 8) * 32 + r % 8 * 4 + lane % 8 / 2] =
                INT8 ? make_uint4(half_pair(x0, x2), half_pair(x1, x3), half_pair(x4, x6), half_pair(x5, x7))
                     : make_uint4(half_pair(x0, x1), half_pair(x2, x3), half_pair(x4, x5), half_pair(x6, x7));
        const float sum = INT8 ? warp_sum(((x0 + x1) + (x2 + x3)) + ((x4 + x5) + (x6 + x7))) : 0.f;
        if (lane == 0) {
            s_factor[r] = p.scale * 1.44269504088896341f * fp16_factor_inverse(e);
            s_bias[r] = sum * (-128.f / 16777216.f);
        }
    }
    __syncthreads();
    // in registers, or read again for each block where the sums need these (D = 256, 16 rows)
    constexpr bool QREG = D * NT <= 256;
    uint4 q[QREG ? J * 2 : 1][NT];
#pragma unroll
    for (int i = 0; i < (QREG ? J * 2 : 1); ++i)
#pragma unroll
        for (int m = 0; m < NT; ++m) q[i][m] = s_q[(i * NT + m) * 32 + lane];

    // this lane's columns: query rows m * 8 + 2t + e
    float factor[NT][2], bias[NT][2], top[NT][2], l_round[NT][2], l_sum[NT][2], o[NT][MT][4];
    int here[NT][2];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = m * 8 + 2 * t + e;
            factor[m][e] = s_factor[r] * UNIT;
            bias[m][e] = INT8 ? s_bias[r] : 0.f;
            // the window counts from the position even where that is beyond the table; before 0 is before 0
            here[m][e] = (int)max(base + (r0 + min(r, live - 1)) / share, -1ll);
            top[m][e] = -INFINITY;
            l_round[m][e] = l_sum[m][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) o[m][i][0] = o[m][i][1] = o[m][i][2] = o[m][i][3] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) s_spoilt[m * 2 + e][threadIdx.x] = 0;
    }
    bool spoilt = false;
    // blocks inside [clear_lo, clear_hi) are seen whole by every row
    const long long clear_lo = p.window > 0 ? max(0ll, base + q_hi - p.window + 1) : 0, clear_hi = min(base + q_lo + 1, (long long)cap);

    const int steps = (s_hi - s_lo + kW * U - 1) / (kW * U);
    for (int it = 0; it < steps; ++it) {
        cp_async_wait<1>();
        const uint8_t *stage = ring + (it & 1) * kStage;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int pos = (s_lo + (it * kW + warp) * U + u) * 16;
            if (ok[u] && q_lo != q_hi && (pos < clear_lo || pos + 16 > clear_hi) &&
                note_spoilt<D, INT8, NT>(ring + (it & 1) * kStage + u * 32 * D + 16 * D, vs[u], &s_spoilt[0][threadIdx.x], pos, base, r0,
                                         share, live, lo, end, p.window)) {
                spoilt = true;
                if (!(fabsf(vs[u]) < INFINITY)) vs[u] = 0.f;
            }
        }

        float s[U][NT][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!ok[u]) {
#pragma unroll
                for (int m = 0; m < NT; ++m) s[u][m][0] = s[u][m][1] = s[u][m][2] = s[u][m][3] = -INFINITY;
                continue;
            }
            float d[NT][4], d2[NT][4];   // two chains of products
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint4 x = *(const uint4 *)(stage + u * 32 * D + j * 1024), y = *(const uint4 *)(stage + u * 32 * D + j * 1024 + 512);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a0, a1, a2, a3;
                    key_operands<INT8>(xw[i], a0, a2);
                    key_operands<INT8>(yw[i], a1, a3);
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        const uint4 v = QREG ? q[(j * 2 + i / 2) % (QREG ? J * 2 : 1)][m] : s_q[((j * 2 + i / 2) * NT + m) * 32 + lane];
                        const uint32_t b0 = i % 2 ? v.z : v.x, b1 = i % 2 ? v.w : v.y;
                        if (j == 0 && i == 0)
                            mma_f16_from(d[m], a0, a1, a2, a3, b0, b1, bias[m][0], bias[m][1]);
                        else if (j == 0 && i == 1)
                            mma_f16_first(d2[m], a0, a1, a2, a3, b0, b1);
                        else
                            mma_f16(i % 2 ? d2[m] : d[m], a0, a1, a2, a3, b0, b1);
                    }
                }
            }
            const int pos = (s_lo + (it * kW + warp) * U + u) * 16;
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[u][m][e] = (d[m][e] + d2[m][e]) * (factor[m][e % 2] * ks[u]);
            if (pos < clear_lo || pos + 16 > clear_hi) {
#pragma unroll
                for (int m = 0; m < NT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = pos + g + e / 2 * 8;
                        if (at > here[m][e % 2] || at >= end || (p.window > 0 && here[m][e % 2] - at >= p.window)) s[u][m][e] = -INFINITY;
                    }
            }
        }

        // a new reference where a score is over 8 above the old one
        bool up = false;
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float most = fmaxf(s[0][m][e], s[0][m][e + 2]);
#pragma unroll
                for (int u = 1; u < U; ++u) most = fmaxf(most, fmaxf(s[u][m][e], s[u][m][e + 2]));
                up |= most > top[m][e] + 8.f;
            }
        if (__any_sync(~0u, up)) {
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                float keep[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float most = fmaxf(s[0][m][e], s[0][m][e + 2]);
#pragma unroll
                    for (int u = 1; u < U; ++u) most = fmaxf(most, fmaxf(s[u][m][e], s[u][m][e + 2]));
                    most = fmaxf(most, __shfl_xor_sync(~0u, most, 4));
                    most = fmaxf(most, __shfl_xor_sync(~0u, most, 8));
                    most = fmaxf(most, __shfl_xor_sync(~0u, most, 16));
                    most = fmaxf(most, top[m][e]);
                    keep[e] = most == top[m][e] ? 1.f : exp2_fast(top[m][e] - most);
                    top[m][e] = most;
                    l_round[m][e] *= keep[e];
                    l_sum[m][e] *= keep[e];
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) o[m][i][0] *= keep[0], o[m][i][1] *= keep[1], o[m][i][2] *= keep[0], o[m][i][3] *= keep[1];
            }
        }

#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!ok[u]) continue;
            uint32_t b0[NT], b1[NT];
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float from = top[m][e % 2] == -INFINITY ? 0.f : top[m][e % 2] - kHeadroom;   // no token of the row yet
                    w[e] = exp2_fast(s[u][m][e] - from);
                }
                l_sum[m][0] += w[0] + w[2];
                l_sum[m][1] += w[1] + w[3];
                b0[m] = transpose_8x8(half_pair(w[0], w[1]));
                b1[m] = transpose_8x8(half_pair(w[2], w[3]));
                float l[4];
                constexpr uint32_t ones = 0x3c003c00u;
                mma_f16_first(l, ones, ones, ones, ones, b0[m], b1[m]);
                l_round[m][0] += l[0];
                l_round[m][1] += l[1];
            }
            const float scale = vs[u];
            const uint8_t *values = stage + u * 32 * D + 16 * D;
#pragma unroll
            for (int j = 0; j < (D < 128 ? 1 : D / 128); ++j) {
                uint32_t w[4][E / 4];   // words of the four tokens
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (D < 128) {
                        const uint2 v = *(const uint2 *)(values + i / 2 * 512 + i % 2 * 8);
                        w[i][0] = v.x, w[i][1] = v.y;
                    } else {
                        const uint4 v = *(const uint4 *)(values + (j * 4 + i) * 512);
                        w[i][0] = v.x, w[i][1] = v.y, w[i][2 % (E / 4)] = v.z, w[i][3 % (E / 4)] = v.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    uint32_t lo4[4], hi4[4];
                    value_operands<INT8>(w[0][i], w[1][i], lo4);
                    value_operands<INT8>(w[2][i], w[3][i], hi4);
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int m = 0; m < NT; ++m) {
                            float d[4];
                            mma_f16_first(d, lo4[half * 2], lo4[half * 2 + 1], hi4[half * 2], hi4[half * 2 + 1], b0[m], b1[m]);
                            float(&acc)[4] = o[m][j * 8 + i * 2 + half];
                            fma_pair(acc[0], acc[1], scale, d[0], d[1]);
                            fma_pair(acc[2], acc[3], scale, d[2], d[3]);
                        }
                }
            }
        }
        advance();
        load(it + 2, n_place, n_ks, n_vs, n_ok);   // into the slot just read, by the lane that read it
        cp_async_commit();
        fetch(it + 3, n_place);
    }

    // Join the warps.  Their sums, relative to the CTA's maximum, take the rings' place, columns
    // c of lane group g at word (8c + g) ^ (8 (r / 2 % 4)) of their piece of 128, which keeps a
    // warp's stores off each other's banks.
    cp_async_wait<0>();
    if (spoilt) {
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t columns = s_spoilt[m * 2 + e % 2][threadIdx.x];
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    if (columns >> (i * 2 + e / 2) & 1) o[m][i][e] = NAN;
            }
    }
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = l_sum[m][e];
            l += __shfl_xor_sync(~0u, l, 4);
            l += __shfl_xor_sync(~0u, l, 8);
            l += __shfl_xor_sync(~0u, l, 16);
            if (g == 0) {
                const int r = m * 8 + 2 * t + e;
                s_stat[warp][0][r] = top[m][e], s_stat[warp][1][r] = l_round[m][e], s_stat[warp][2][r] = l;
            }
        }
    __syncthreads();
    auto weight = [](float m, float most) { return m == -INFINITY ? 0.f : exp2_fast(m - most); };
    float *sums = (float *)smem;   // [warp][R][D]
#pragma unroll
    for (int m = 0; m < NT; ++m) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = m * 8 + 2 * t + e;
            float most = s_stat[0][0][r];
#pragma unroll
            for (int w = 1; w < kW; ++w) most = fmaxf(most, s_stat[w][0][r]);
            f[e] = weight(top[m][e], most);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = i % 8 * 2 + e / 2, r = m * 8 + 2 * t + e % 2;
                sums[(warp * R + r) * D + i / 8 * 128 + ((col * 8 + g) ^ (t * 8))] = o[m][i][e] * f[e % 2];
            }
    }
    if (threadIdx.x < R) {
        const int r = threadIdx.x;
        float most = s_stat[0][0][r], l = 0.f, e = 0.f;
#pragma unroll
        for (int w = 1; w < kW; ++w) most = fmaxf(most, s_stat[w][0][r]);
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            const float f = weight(s_stat[w][0][r], most);
            l = fmaf(f, s_stat[w][1][r], l), e = fmaf(f, s_stat[w][2][r], e);
        }
        s_total[r] = make_float4(most, l, e, 0.f);
    }
    __syncthreads();
    float4 *sums4 = (float4 *)sums;
    for (int i = threadIdx.x; i < live * D / 4; i += kW * 32) {
        float4 v = sums4[i];
#pragma unroll
        for (int w = 1; w < kW; ++w) {
            const float4 x = sums4[w * R * D / 4 + i];
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        sums4[i] = v;
    }
    // a word's column, and what becomes of a row's sum and statistics
    auto column = [&](int r, int word) {
        const int x = word % 128 ^ (r / 2 % 4 * 8);
        return word / 128 * 128 + x % 8 * E + x / 8;
    };
    auto finish = [&](int r, int word, float4 v, float l) {
        const int row = r0 + r, d = column(r, word);   // the next three words are the next three lane groups
        const float f = l == 0.f ? 0.f : 1.f / l;
        uint16_t *out = p.out + ((long long)(row0 + row / share) * p.heads + h * share + row % share) * D + d;
        out[0] = bf16_bits(v.x * f), out[E] = bf16_bits(v.y * f), out[2 * E] = bf16_bits(v.z * f), out[3 * E] = bf16_bits(v.w * f);
    };
    auto finish_lse = [&](int r, float most, float e) {
        const int row = r0 + r;
        if (p.lse)
            p.lse[(long long)(row0 + row / share) * p.heads + h * share + row % share] =
                e == 0.f ? -INFINITY : (most - kHeadroom + log2f(e)) * 0.69314718055994531f;
    };
    if (csize == 1 && clusters == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < live * D / 4; i += kW * 32) finish(i * 4 / D, i * 4 % D, sums4[i], s_total[i * 4 / D].y);
        if (threadIdx.x < live) finish_lse(threadIdx.x, s_total[threadIdx.x].x, s_total[threadIdx.x].z);
        return;
    }

    // Join the cluster: every CTA takes a slice of a row's words, [crank * width, + width).
    // Each thread reads the CTAs' statistics of its row beside their sums, and weighs them itself.
    struct Joined {
        float4 v;
        float most, l, e;
    };
    auto take = [&](Joined &j, const auto &stat, const auto &x) {   // parties that are not there: most = -inf, zeros
        constexpr int N = sizeof(stat) / sizeof(float4);
        float most = j.most;
#pragma unroll
        for (int k = 0; k < N; ++k) most = fmaxf(most, stat[k].x);
        const float f = weight(j.most, most);
        j.v.x *= f, j.v.y *= f, j.v.z *= f, j.v.w *= f, j.l *= f, j.e *= f, j.most = most;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float f = weight(stat[k].x, most);
            j.v.x = fmaf(f, x[k].x, j.v.x), j.v.y = fmaf(f, x[k].y, j.v.y), j.v.z = fmaf(f, x[k].z, j.v.z), j.v.w = fmaf(f, x[k].w, j.v.w);
            j.l = fmaf(f, stat[k].y, j.l), j.e = fmaf(f, stat[k].z, j.e);
        }
    };
    const Joined nothing = {make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f, 0.f};
    const float4 absent = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    const int width = D / csize, quads = live * width / 4, row_shift = 31 - __clz(width / 4);
    const long long stride = partial_floats(D, R);
    float *partial = p.partial + item * (p.splits / csize) * stride;
    auto end_of = [&](int r, int word, bool first, const Joined &j) {
        finish(r, word, j.v, j.l);
        if (crank == 0 && first) finish_lse(r, j.most, j.e);
    };
    cluster_sync();
    for (int i = threadIdx.x; i < quads; i += kW * 32) {
        const int r = i >> row_shift, in_row = i - (r << row_shift), word = crank * width + in_row * 4;
        float4 stat[kMaxCluster], x[kMaxCluster];
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            stat[k] = absent, x[k] = nothing.v;
            if (k < csize) stat[k] = cluster_load4((const float *)(s_total + r), k), x[k] = cluster_load4(sums + r * D + word, k);
        }
        Joined j = nothing;
        take(j, stat, x);
        if (clusters == 1) {
            end_of(r, word, in_row == 0, j);
        } else {
            *(float4 *)(partial + ck * stride + r * D + word) = j.v;
            if (in_row == 0) *(float4 *)(partial + ck * stride + R * D + (crank * R + r) * 4) = make_float4(j.most, j.l, j.e, 0.f);
        }
    }
    cluster_arrive();   // this CTA has read the others' sums
    if (clusters == 1) {
        cluster_wait();   // the others may still be reading this CTA's
        return;
    }

    // Join the clusters: the last one to arrive, per slice of columns.  The barrier and the
    // ticket's release carry this CTA's sums, its acquire and the barrier the others'.
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t *ticket = p.tickets + item * kMaxCluster + crank;
        s_last = atom_add_acq_rel(ticket, 1) == (uint32_t)clusters - 1;
        if (s_last) *ticket = 0;
    }
    __syncthreads();
    cluster_wait();   // the others may still be reading this CTA's sums
    if (!s_last) return;
    // `lanes` threads for four words, each with every lanes-th cluster, some at a time
    constexpr int FEW = D == 256 ? 16 : 8;
    int lanes = 1;
    while (lanes < 32 && quads * lanes * 2 <= kW * 32) lanes *= 2;
    const int from = threadIdx.x % lanes;
    for (int q0 = 0; q0 < quads; q0 += kW * 32 / lanes) {
        const int i = q0 + threadIdx.x / lanes, r = i < quads ? i >> row_shift : 0, in_row = i - (r << row_shift), word = crank * width + in_row * 4;
        const float *src = partial + r * D + (i < quads ? word : 0), *src_stat = partial + R * D + (crank * R + r) * 4;
        Joined j = nothing;
        for (int k0 = from; k0 < clusters; k0 += FEW * lanes) {
            float4 stat[FEW], x[FEW];
#pragma unroll
            for (int k = 0; k < FEW; ++k) {
                const int at = k0 + k * lanes;
                stat[k] = absent, x[k] = nothing.v;
                if (at < clusters) stat[k] = __ldcg((const float4 *)(src_stat + at * stride)), x[k] = __ldcg((const float4 *)(src + at * stride));
            }
            take(j, stat, x);
        }
        for (int o = 1; o < lanes; o *= 2) {
            const float4 stat[1] = {make_float4(__shfl_xor_sync(~0u, j.most, o), __shfl_xor_sync(~0u, j.l, o), __shfl_xor_sync(~0u, j.e, o), 0.f)};
            const float4 x[1] = {make_float4(__shfl_xor_sync(~0u, j.v.x, o), __shfl_xor_sync(~0u, j.v.y, o), __shfl_xor_sync(~0u, j.v.z, o),
                                             __shfl_xor_sync(~0u, j.v.w, o))};
            take(j, stat, x);
        }
        if (i < quads && from == 0) end_of(r, word, in_row == 0, j);
    }
}

template <int D, bool INT8, int NT> cudaError_t launch(const KvAttentionParams &p, const KvAttentionPlan &plan, cudaStream_t s)
{
    const size_t smem = ring_bytes(D, NT) + D / 64 * 2 * NT * 512;
    cudaError_t e = allow_smem((const void *)k_kv_attention<D, INT8, NT>, smem);
    if (e != cudaSuccess) return e;
    return launch_clusters(k_kv_attention<D, INT8, NT>, dim3(plan.splits, p.c.kv_heads * plan.row_tiles, p.c.batch), dim3(kW * 32),
                           plan.cluster, smem, s, p);
}

template <int D> cudaError_t launch_dim(const KvAttentionParams &p, const KvAttentionPlan &plan, cudaStream_t s)
{
    if (p.c.format == MTP_KV_INT8) return plan.tiles8 == 1 ? launch<D, true, 1>(p, plan, s) : launch<D, true, 2>(p, plan, s);
    return plan.tiles8 == 1 ? launch<D, false, 1>(p, plan, s) : launch<D, false, 2>(p, plan, s);
}

}  // namespace

KvAttentionPlan kv_attention_plan(const KvParams &c, int heads, int window, int max_len)
{
    KvAttentionPlan plan{};
    const long long longest_q = c.starts ? c.max_tokens : c.tokens / c.batch, rows = longest_q * (heads / c.kv_heads);
    plan.tiles8 = rows <= 8 ? 1 : 2;
    const int R = plan.tiles8 * 8;
    plan.row_tiles = (int)((rows + R - 1) / R);
    plan.items = (long long)c.batch * c.kv_heads * plan.row_tiles;
    const long long cap = (long long)c.table_width * c.page_tokens;
    long long seen = max_len > 0 ? std::min<long long>(max_len, cap) : cap;
    if (window > 0) seen = std::min(seen, window + longest_q - 1);
    const long long slots = (long long)sm_count() * ctas_per_sm(c.dim, plan.tiles8), blocks = seen / 16 + 1;
    // CTAs of an item.  Alike items (one sequence, or a window of all): what fits at once, less
    // the 3 % that whole clusters leave empty, or four rounds where even one each is half of
    // that.  Unlike ones: one cluster each, in up to four rounds, or more clusters where a round
    // and a quarter has room (32 heads on 8, D = 128, up to 8191 tokens: 8 sequences with 4, 8,
    // 16, 24 CTAs an item 32.5, 24.4, 29.5, 28.5 us; 24 sequences with 2, 4, 8, 16: 69, 61, 59, 73
    // us; 4 sequences with 8, 16, 24, 32: 16.6, 14.4, 14.3, 14.4 us; the window of 512, 64 items,
    // with 2, 4, 8: 13.9, 12.7, 18.6 us).  At D = 256, whose joins are larger, clusters of four
    // where these fill two thirds of the places (80 items of up to 4434 tokens with 2, 4, 8: 53,
    // 38, 41 us; 37 items of up to 5889 with 4, 8, 16: 37, 27, 31 us).
    const bool alike = c.batch == 1 || window > 0;
    const long long fit = slots * 97 / 100 / plan.items, loose = slots * 5 / 4 / plan.items, rounds = 4 * slots / plan.items;
    const long long one = c.dim == 256 && plan.items * 6 >= slots ? 4 : 8;
    long long splits = alike ? (plan.items >= slots / 2 ? rounds : fit) : loose >= 16 ? loose : std::min(rounds, one);
    // at least kMinBlocks each; a first cluster costs little, so a block for each warp is
    // enough for that where it fits at once
    const long long most = std::max((blocks + kMinBlocks - 1) / kMinBlocks, std::min({8ll, fit, (blocks + kW - 1) / kW}));
    splits = std::max(1ll, std::min({splits, most, (long long)kMaxSplits}));
    const long long up = alike ? 0 : 1;
    plan.cluster = splits >= 8 - 2 * up ? 8 : splits >= 4 - up ? 4 : splits >= 2 ? 2 : 1;
    splits = std::max<long long>(plan.cluster, splits / plan.cluster * plan.cluster);
    // without tickets for every item there is one cluster for each
    if (plan.items * kMaxCluster > MTP_KV_WORKSPACE_ZEROED / 4) splits = plan.cluster;
    plan.splits = (int)splits;
    if (splits > plan.cluster)
        plan.partial_floats = (size_t)plan.items * (splits / plan.cluster) * partial_floats(c.dim, R);
    return plan;
}

cudaError_t launch_kv_attention(KvAttentionParams p, const KvAttentionPlan &plan, cudaStream_t s)
{
    const uint32_t page_blocks = p.c.page_tokens / 16;
    p.page_magic = page_blocks == 1 ? 0 : (uint32_t)(0xffffffffu / page_blocks) + 1;   // exact below 2^26 blocks of 16
    p.row_tiles = plan.row_tiles;
    p.splits = plan.splits;
    return p.c.dim == 64 ? launch_dim<64>(p, plan, s) : p.c.dim == 128 ? launch_dim<128>(p, plan, s) : launch_dim<256>(p, plan, s);
}

}  // namespace mtp
