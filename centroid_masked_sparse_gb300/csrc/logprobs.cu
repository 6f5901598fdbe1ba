// Log probabilities of given tokens, entropy and largest alternatives of rows of logits,
// and the gradient of the former two.
#include <algorithm>

#include "lm_ops.h"

namespace mtp {

namespace {

constexpr int kLpThreads = 256;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

template <typename T> __device__ __forceinline__ float logit_value(T v);
template <> __device__ __forceinline__ float logit_value(float v) { return v; }
template <> __device__ __forceinline__ float logit_value(uint16_t v) { return bf16_value(v); }

// (larger logit, then lower id) as one unsigned key; 0 for a masked token.
__device__ __forceinline__ unsigned long long top_key(float v, int id)
{
    return v == -INFINITY ? 0ull : argmax_key(v, id);
}

// One CTA per row.  Terms are e = 2^d of d = (x - max x) * c, c = log2(e) / temperature, with
// the maximum subtracted first: x * c may leave fp32's range, and its rounding would grow
// with x.  s = sum e and t = sum e * d give ln sum and entropy.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) k_token_logprobs(LogprobParams p)
{
    __shared__ float s_a[kLpThreads / 32], s_b[kLpThreads / 32];
    __shared__ int s_n[kLpThreads / 32];
    __shared__ unsigned long long s_k[kLpThreads / 32];
    const int row = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const T *x = (const T *)p.logits + row * p.ld;
    const float c = p.factor * kLog2e;
    const int given = p.tokens ? __ldg(p.tokens + row) : -1;
    const bool has = given >= 0 && given < p.vocab;
    const float mine = has ? logit_value(x[given]) : 0.f;

    float top = -INFINITY;
    int before = 0;
    for (int i = threadIdx.x; i < p.vocab; i += kLpThreads) {
        const float v = logit_value(x[i]);
        top = fmaxf(top, v);
        before += v > mine || (v == mine && i < given);
    }
    for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        before += __shfl_xor_sync(~0u, before, o);
    }
    if (lane == 0) s_a[warp] = top, s_n[warp] = before;
    __syncthreads();
    before = 0;
    for (int w = 0; w < kLpThreads / 32; ++w) top = fmaxf(top, s_a[w]), before += s_n[w];
    __syncthreads();
    const float m = top == -INFINITY ? 0.f : top;
    float s = 0.f, t = 0.f;
    for (int i = threadIdx.x; i < p.vocab; i += kLpThreads) {
        const float d = (logit_value(x[i]) - m) * c, e = exp2_fast(d);
        s += e;
        if (e > 0.f) t = fmaf(e, d, t);
    }
    s = warp_sum(s), t = warp_sum(t);
    if (lane == 0) s_a[warp] = s, s_b[warp] = t;
    __syncthreads();
    s = t = 0.f;
    for (int w = 0; w < kLpThreads / 32; ++w) s += s_a[w], t += s_b[w];
    const float lns = logf(s);
    if (threadIdx.x == 0) {
        if (p.lse) p.lse[row] = fmaf(m, p.factor, lns);
        if (p.entropy) p.entropy[row] = s == 0.f ? 0.f : lns - t / s * kLn2;
        if (p.logprob)
            p.logprob[row] = !has ? 0.f : mine == -INFINITY ? -INFINITY + s * 0.f : fmaf(mine - m, p.factor, -lns);
        if (p.rank) p.rank[row] = has ? before : -1;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < p.top; ++k) {
        unsigned long long best = 0;
        for (int i = threadIdx.x; i < p.vocab; i += kLpThreads) {
            const unsigned long long key = top_key(logit_value(x[i]), i);
            if (key < last && key > best) best = key;
        }
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(~0u, best, o));
        __syncthreads();
        if (lane == 0) s_k[warp] = best;
        __syncthreads();
        for (int w = 0; w < kLpThreads / 32; ++w) best = max(best, s_k[w]);
        last = best;
        if (threadIdx.x == 0) {
            int id;
            float v;
            decode_argmax_key(best, &id, &v);
            p.top_ids[(long long)row * p.top + k] = id;
            if (p.top_logprobs)
                p.top_logprobs[(long long)row * p.top + k] = best == 0 ? -INFINITY + s * 0.f : fmaf(v - m, p.factor, -lns);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) k_token_logprobs_backward(LogprobGradParams p)
{
    const int row = blockIdx.x;
    const T *x = (const T *)p.logits + row * p.ld;
    T *g = (T *)p.grad + row * p.ld_grad;
    const float lse = __ldg(p.lse + row);
    const int given = p.tokens ? __ldg(p.tokens + row) : -1;
    const bool has = given >= 0 && given < p.vocab;
    const float gl = p.grad_logprob && has ? __ldg(p.grad_logprob + row) : 0.f;
    const float ge = p.grad_entropy ? __ldg(p.grad_entropy + row) : 0.f;
    const float h = p.grad_entropy ? __ldg(p.entropy + row) : 0.f;
    for (long long i = blockIdx.y * kLpThreads + threadIdx.x; i < p.vocab; i += gridDim.y * kLpThreads) {
        const float v = logit_value(x[i]);
        float r = 0.f;
        if (v != -INFINITY) {
            const float d = fmaf(v, p.factor, -lse), e = exp2_fast(d * kLog2e);
            r = ((i == given ? gl : 0.f) - e * (gl + ge * (d + h))) * p.factor;
        }
        if constexpr (sizeof(T) == 2)
            g[i] = bf16_bits(r);
        else
            g[i] = r;
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams &p, bool bf16, cudaStream_t s)
{
    if (bf16)
        k_token_logprobs<uint16_t><<<p.rows, kLpThreads, 0, s>>>(p);
    else
        k_token_logprobs<float><<<p.rows, kLpThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_token_logprobs_backward(const LogprobGradParams &p, bool bf16, cudaStream_t s)
{
    const dim3 grid(p.rows, (unsigned)std::min((p.vocab + kLpThreads * 16ll - 1) / (kLpThreads * 16), 65535ll));
    if (bf16)
        k_token_logprobs_backward<uint16_t><<<grid, kLpThreads, 0, s>>>(p);
    else
        k_token_logprobs_backward<float><<<grid, kLpThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mtp
