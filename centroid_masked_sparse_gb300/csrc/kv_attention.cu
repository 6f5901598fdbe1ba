// Attention of one or a few query tokens per sequence over the paged 8-bit cache.
#include "lm_ops.h"

namespace mtp {

namespace {

constexpr int kAttnThreads = 128;

// One CTA per (query token, head); each warp takes every fourth cached token and keeps a
// running maximum, sum and weighted value; the warps' results are joined at the end.
template <int D>
__global__ void __launch_bounds__(kAttnThreads) k_kv_attention(KvAttentionParams p)
{
    constexpr int E = D / 32, W = kAttnThreads / 32;
    const KvParams &c = p.c;
    __shared__ float s_m[W], s_l[W], s_o[W][D];
    const int b = blockIdx.y, head = blockIdx.z, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int row0, n;
    kv_rows(c, b, &row0, &n);
    if ((int)blockIdx.x >= n) return;
    const long long row = row0 + blockIdx.x;
    const int h = head / (p.heads / c.kv_heads);
    const long long P = c.page_tokens;
    long long length = __ldg(c.lengths + b);
    const long long here = length - n + blockIdx.x;
    if (length < 0 || length > c.table_width * P) {
        if (c.err && threadIdx.x == 0) atomicOr(c.err, MTP_DEVERR_PAGE);
    }
    const long long first = p.window > 0 ? max(0ll, here - p.window + 1) : 0, end = min(here + 1, c.table_width * P);

    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = bf16_value(p.q[row * p.q_token + head * p.q_head + e * 32 + lane]);
    for (long long t = first + warp; t < end; t += W) {
        const int page = __ldg(c.table + b * c.ld_table + t / P);
        if (page < 0 || page >= c.pages) {
            if (c.err && lane == 0) atomicOr(c.err, MTP_DEVERR_PAGE);
            continue;
        }
        const long long ph = (long long)page * c.kv_heads + h, at = (ph * P + t % P) * D;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], kv_value(c.k_codes[at + e * 32 + lane], c.format), s);
        s = warp_sum(s) * p.scale * c.k_scales[ph];
        const float up = fmaxf(m, s), keep = up == -INFINITY ? 1.f : expf(m - up), w = up == -INFINITY ? 0.f : expf(s - up);
        m = up;
        l = l * keep + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * c.v_scales[ph] * kv_value(c.v_codes[at + e * 32 + lane], c.format);
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][e * 32 + lane] = o[e];
    __syncthreads();
    m = s_m[0];
    for (int w = 1; w < W; ++w) m = fmaxf(m, s_m[w]);
    l = 0.f;
    for (int w = 0; w < W; ++w) l += m == -INFINITY ? s_l[w] : expf(s_m[w] - m) * s_l[w];
    for (int d = threadIdx.x; d < D; d += kAttnThreads) {
        float v = 0.f;
        for (int w = 0; w < W; ++w) v += m == -INFINITY ? 0.f : expf(s_m[w] - m) * s_o[w][d];
        p.out[(row * p.heads + head) * D + d] = bf16_bits(l == 0.f ? 0.f : v / l);
    }
    if (p.lse && threadIdx.x == 0) p.lse[row * p.heads + head] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttentionParams &p, cudaStream_t s)
{
    const int longest = p.c.starts ? p.c.max_tokens : p.c.tokens / p.c.batch;
    const dim3 grid(longest, p.c.batch, p.heads);
    if (p.c.dim == 64)
        k_kv_attention<64><<<grid, kAttnThreads, 0, s>>>(p);
    else if (p.c.dim == 128)
        k_kv_attention<128><<<grid, kAttnThreads, 0, s>>>(p);
    else
        k_kv_attention<256><<<grid, kAttnThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mtp
