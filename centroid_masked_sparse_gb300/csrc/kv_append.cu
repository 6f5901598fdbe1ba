// New keys and values into the paged 8-bit cache: one scale per (page, kv head), raised
// when a new token needs it, in which case the page's earlier codes are rounded again.
//
// One CTA per (block that the call reaches, kv head, keys or values): it holds the block's new
// values in registers between the search for the largest and the rounding, so that they are
// read once; only blocks of more than 16384 new values are read twice.
//
// The rounding asks for IEEE divisions, x / scale.  A product with the reciprocal is within
// 2^-22 of the quotient (two roundings against one), so where the products a little below and
// a little above round to the same code, the quotient does too; else, about once in ten
// thousand values, the division is done.  Non-finite values and scales beyond 2^+-100 take the
// plain way for their block.
//
// Bound by latency for single tokens (64 of them, 8 heads of 128, take 3.0 us in a graph) and
// by instructions for prompts (2 x 2049 tokens: 10.9 us in a graph, with a division for every
// value 15.5, with two readings of them 40).
#include <algorithm>

#include "lm_ops.h"

namespace mtp {

namespace {

constexpr int kAppendThreads = 256;   // at most
constexpr int kAppendVecs = 8;        // vectors of 8 values that a thread holds

// A finite value of a bf16 input: NaN counts as 0, infinities as the largest finite bf16.
__device__ __forceinline__ float finite_bf16(float v)
{
    return v == v ? fminf(fmaxf(v, -3.38953139e38f), 3.38953139e38f) : 0.f;
}

struct Eight {
    float v[8];
};
__device__ __forceinline__ Eight finite_values(const uint4 &u)
{
    return Eight{finite_bf16(bf_lo(u.x)), finite_bf16(bf_hi(u.x)), finite_bf16(bf_lo(u.y)), finite_bf16(bf_hi(u.y)),
                 finite_bf16(bf_lo(u.z)), finite_bf16(bf_hi(u.z)), finite_bf16(bf_lo(u.w)), finite_bf16(bf_hi(u.w))};
}

// blockIdx.x counts a sequence's blocks from its first new one.
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(KvAppendParams p)
{
    const KvParams &c = p.c;
    __shared__ uint32_t s_max[kAppendThreads / 32];
    const int b = blockIdx.y, h = blockIdx.z >> 1, threads = blockDim.x;
    const bool values = blockIdx.z & 1;
    wait_for_previous();
    const int before = __ldg(c.lengths + b);
    int row0, n;
    kv_rows(c, b, &row0, &n);
    if (n <= 0) return;
    if (before < 0) {
        if (c.err && threadIdx.x == 0) atomicOr(c.err, MTP_DEVERR_PAGE);
        return;
    }
    // block `at` of the sequence holds its positions [at * P, (at + 1) * P); new tokens are
    // positions [before, before + n)
    const int P = c.page_tokens;
    const long long at = before / P + blockIdx.x;
    const long long lo = max((long long)before, at * P), hi = min((long long)before + n, (at + 1) * P);
    if (lo >= hi) return;
    int page = -1;
    if (at < c.table_width) page = __ldg(c.table + b * c.ld_table + at);
    if (page < 0 || page >= c.pages) {
        if (c.err && threadIdx.x == 0) atomicOr(c.err, MTP_DEVERR_PAGE);
        return;
    }
    const int D = c.dim, shift = D == 64 ? 3 : D == 128 ? 4 : 5;   // vectors of a token
    const int first = (int)(lo - at * P), vecs = (int)(hi - lo) << shift;
    const uint16_t *x = values ? p.v + h * p.v_head : p.k + h * p.k_head;
    const long long stride = values ? p.v_token : p.k_token;
    x += (row0 + (lo - before)) * stride;
    const long long ph = (long long)page * c.kv_heads + h;
    uint2 *codes = (uint2 *)((values ? c.v_codes : c.k_codes) + ph * P * D);
    float *scale_at = (values ? c.v_scales : c.k_scales) + ph;
    const float old = first > 0 ? *scale_at : 0.f;
    auto load = [&](int i) { return ld_ro16(x + (i >> shift) * stride + (i & ((1 << shift) - 1)) * 8); };

    uint4 held[kAppendVecs];
    const bool holds = vecs <= kAppendVecs * threads;
    if (holds) {
#pragma unroll
        for (int k = 0; k < kAppendVecs; ++k)
            held[k] = (int)threadIdx.x + k * threads < vecs ? load(threadIdx.x + k * threads) : make_uint4(0, 0, 0, 0);
    }
    auto each = [&](auto f) {
        if (holds) {
#pragma unroll
            for (int k = 0; k < kAppendVecs; ++k)
                if ((int)threadIdx.x + k * threads < vecs) f(threadIdx.x + k * threads, held[k]);
        } else {
#pragma unroll 2
            for (int i = threadIdx.x; i < vecs; i += threads) f(i, load(i));
        }
    };
    // the largest magnitude, as bits: these are ordered like the values, non-finite ones last
    auto largest = [&](uint32_t mine) {
        mine = __reduce_max_sync(~0u, mine);
        if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = mine;
        __syncthreads();
        for (int w = 0; w < threads / 32; ++w) mine = max(mine, s_max[w]);
        return mine;
    };
    uint32_t most = 0;
    each([&](int, const uint4 &u) {
        most = __vmaxu2(most, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
    });
    uint32_t top = largest(max(most >> 16, most & 0xffffu));
    const bool odd = top >= 0x7f80u;   // NaN or infinity
    if (odd) {
        most = 0;
        each([&](int, const uint4 &u) {
            const Eight e = finite_values(u);
#pragma unroll
            for (int k = 0; k < 8; ++k) most = max(most, __float_as_uint(fabsf(e.v[k])) >> 16);
        });
        __syncthreads();
        top = largest(most);
    }
    const float scale = fmaxf(old, __fdiv_rn(bf16_value((uint16_t)top), c.format == MTP_KV_INT8 ? 127.f : 448.f));
    if (threadIdx.x == 0) *scale_at = scale;   // every thread has read the old one
    if (scale != old) {
        const float ratio = scale > 0.f ? __fdiv_rn(old, scale) : 0.f;
        for (int i = threadIdx.x; i < first << shift; i += threads) {
            uint2 u = codes[i];
            auto again = [&](uint32_t w) {
                return kv_codes(kv_value(w, c.format) * ratio, kv_value(w >> 8, c.format) * ratio, kv_value(w >> 16, c.format) * ratio,
                                kv_value(w >> 24, c.format) * ratio, c.format);
            };
            u.x = again(u.x), u.y = again(u.y);
            codes[i] = u;
        }
    }
    uint2 *out = codes + (first << shift);
    auto divided = [&](float x, float y, float z, float w) {
        return kv_codes(__fdiv_rn(x, scale), __fdiv_rn(y, scale), __fdiv_rn(z, scale), __fdiv_rn(w, scale), c.format);
    };
    if (odd || !(scale >= 0x1p-100f && scale <= 0x1p100f)) {
        each([&](int i, const uint4 &u) {
            const Eight e = finite_values(u);
            out[i] = scale > 0.f ? make_uint2(divided(e.v[0], e.v[1], e.v[2], e.v[3]), divided(e.v[4], e.v[5], e.v[6], e.v[7])) : make_uint2(0, 0);
        });
    } else {
        const float inverse = __fdiv_rn(1.f, scale), under = inverse * (1.f - 0x1p-21f), over = inverse * (1.f + 0x1p-21f);
        auto four = [&](uint32_t a, uint32_t b) {
            const float x = bf_lo(a), y = bf_hi(a), z = bf_lo(b), w = bf_hi(b);
            const uint32_t code = kv_codes(x * under, y * under, z * under, w * under, c.format);
            if (code == kv_codes(x * over, y * over, z * over, w * over, c.format)) return code;
            return divided(x, y, z, w);
        };
        each([&](int i, const uint4 &u) { out[i] = make_uint2(four(u.x, u.y), four(u.z, u.w)); });
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams &p, cudaStream_t s)
{
    const KvParams &c = p.c;
    const int longest = c.starts ? c.max_tokens : c.tokens / c.batch;
    // a run of n tokens reaches at most (n - 1) / P + 2 blocks, (n + P - 2) / P + 1
    const unsigned blocks = (unsigned)(((long long)longest + c.page_tokens - 2) / c.page_tokens + 1);
    // a vector a thread for few tokens, four where blocks are long; enough for the earlier codes
    const int news = std::min(longest, c.page_tokens) * (c.dim / 8), all = c.page_tokens * (c.dim / 8);
    const int want = std::max(std::min(news, 32), std::max(news / 4, all / 16));
    const int threads = std::min(kAppendThreads, (want + 31) / 32 * 32);
    return launch_dependent(k_kv_append, dim3(blocks, c.batch, 2 * c.kv_heads), dim3(threads), 0, s, p);
}

}  // namespace mtp
