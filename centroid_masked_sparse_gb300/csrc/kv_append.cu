// New keys and values into the paged 8-bit cache: one scale per (page, kv head), raised
// when a new token needs it, in which case the page's earlier codes are rounded again.
#include "lm_ops.h"

namespace mtp {

namespace {

constexpr int kAppendThreads = 128;

// A finite value of a bf16 input: NaN counts as 0, infinities as the largest finite bf16.
__device__ __forceinline__ float finite_bf16(uint16_t h)
{
    const float v = bf16_value(h);
    return v == v ? fminf(fmaxf(v, -3.38953139e38f), 3.38953139e38f) : 0.f;
}

// One CTA per (block that the call reaches, kv head, keys or values); blockIdx.x counts a
// sequence's blocks from its first new one.
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(KvAppendParams p)
{
    const KvParams &c = p.c;
    __shared__ float s_max[kAppendThreads / 32];
    const int b = blockIdx.y, h = blockIdx.z >> 1;
    const bool values = blockIdx.z & 1;
    int row0, n;
    wait_for_previous();
    kv_rows(c, b, &row0, &n);
    const int before = __ldg(c.lengths + b);
    if (n <= 0) return;
    if (before < 0) {
        if (c.err && threadIdx.x == 0) atomicOr(c.err, MTP_DEVERR_PAGE);
        return;
    }
    // block `at` of the sequence holds its positions [at * P, (at + 1) * P); new tokens are
    // positions [before, before + n)
    const long long P = c.page_tokens, at = before / P + blockIdx.x;
    const long long lo = max((long long)before, at * P), hi = min((long long)before + n, (at + 1) * P);
    if (lo >= hi) return;
    int page = -1;
    if (at < c.table_width) page = __ldg(c.table + b * c.ld_table + at);
    if (page < 0 || page >= c.pages) {
        if (c.err && threadIdx.x == 0) atomicOr(c.err, MTP_DEVERR_PAGE);
        return;
    }
    const int D = c.dim, first = (int)(lo - at * P), count = (int)(hi - lo);
    const uint16_t *x = (values ? p.v + h * p.v_head : p.k + h * p.k_head);
    const long long stride = values ? p.v_token : p.k_token;
    x += (row0 + (lo - before)) * stride;
    const long long ph = (long long)page * c.kv_heads + h;
    uint8_t *codes = (values ? c.v_codes : c.k_codes) + ph * P * D;
    float *scale_at = (values ? c.v_scales : c.k_scales) + ph;

    float top = 0.f;
    for (int i = threadIdx.x; i < count * D; i += kAppendThreads)
        top = fmaxf(top, fabsf(finite_bf16(x[i / D * stride + i % D])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = top;
    const float old = first > 0 ? *scale_at : 0.f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) top = fmaxf(top, s_max[w]);
    const float scale = fmaxf(old, __fdiv_rn(top, c.format == MTP_KV_INT8 ? 127.f : 448.f));
    if (threadIdx.x == 0) *scale_at = scale;   // every thread has read the old one
    if (scale != old) {
        const float ratio = scale > 0.f ? __fdiv_rn(old, scale) : 0.f;
        for (int i = threadIdx.x; i < first * D; i += kAppendThreads)
            codes[i] = kv_code(kv_value(codes[i], c.format) * ratio, c.format);
    }
    for (int i = threadIdx.x; i < count * D; i += kAppendThreads) {
        const float v = finite_bf16(x[i / D * stride + i % D]);
        codes[first * D + i] = kv_code(scale > 0.f ? __fdiv_rn(v, scale) : 0.f, c.format);
    }
    let_next_start();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams &p, cudaStream_t s)
{
    const KvParams &c = p.c;
    const int longest = c.starts ? c.max_tokens : c.tokens / c.batch;
    // a run of n tokens reaches at most (n - 1) / P + 2 blocks, (n + P - 2) / P + 1
    const unsigned blocks = (unsigned)(((long long)longest + c.page_tokens - 2) / c.page_tokens + 1);
    return launch_dependent(k_kv_append, dim3(blocks, c.batch, 2 * c.kv_heads), dim3(kAppendThreads), 0, s, p);
}

}  // namespace mtp
