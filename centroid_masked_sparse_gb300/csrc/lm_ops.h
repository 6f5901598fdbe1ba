// Host-side interface between the C ABI of the operators around the head (lm_ops.cu) and
// their kernel files, and the device helpers that these share.
#pragma once

#include "../../include/mtp_lm_ops.h"
#include "internal.h"

namespace mtp {

// ---------------------------------------------------------------------------
// 4-bit products (q4.cu)
// ---------------------------------------------------------------------------
struct Q4Params {
    const uint8_t *codes;    // packed (include/mtp_lm_ops.h), as are scales and zeros
    const uint8_t *scales;
    const uint8_t *zeros;    // or null (8)
    const uint16_t *x;       // bf16 [B, ld_x]
    long long ld_x;
    void *out;               // [B, ld_out] fp32 or bf16
    long long ld_out;
    int M, K, G, group, B;
    int blocks;              // of 64 columns
    int bf16_out;
    float softcap;
};
struct Q4PackParams {
    const uint8_t *codes;    // [M, ld_codes]
    long long ld_codes;      // bytes
    const uint16_t *scales;  // bf16 [M, G]
    const uint8_t *zeros;    // [M, G] or null
    int M, K, G, group, tiles, blocks;
    uint8_t *out_codes, *out_scales, *out_zeros;
};
struct Q4Layout {            // byte offsets of the packed form's parts
    size_t scales, zeros, total;
};
Q4Layout q4_layout(int M, int K, int group, bool zeros);
cudaError_t launch_q4_pack(const Q4PackParams &p, cudaStream_t s);
cudaError_t launch_q4_matvec(const Q4Params &p, cudaStream_t s);
cudaError_t launch_q4_quantize(const uint16_t *w, long long ld_w, int M, int K, int group, uint8_t *codes,
                               long long ld_codes, uint16_t *scales, uint8_t *zeros, cudaStream_t s);

// ---------------------------------------------------------------------------
// The 8-bit cache (kv_append.cu, kv_attention.cu)
// ---------------------------------------------------------------------------
struct KvParams {
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    uint32_t *err;           // device error word or null
    int pages, page_tokens, kv_heads, dim, format;
    const int32_t *table;
    long long ld_table;
    int table_width;
    const int32_t *lengths, *starts;
    int batch, tokens, max_tokens;
};

struct KvAppendParams {
    KvParams c;
    const uint16_t *k, *v;
    long long k_token, k_head, v_token, v_head;   // strides in elements
};
cudaError_t launch_kv_append(const KvAppendParams &p, cudaStream_t s);

struct KvAttentionParams {
    KvParams c;
    const uint16_t *q;
    long long q_token, q_head;
    int heads, window;
    float scale;
    uint16_t *out;
    float *lse;              // or null
};
cudaError_t launch_kv_attention(const KvAttentionParams &p, cudaStream_t s);

// ---------------------------------------------------------------------------
// Token log probabilities (logprobs.cu)
// ---------------------------------------------------------------------------
struct LogprobParams {
    const void *logits;      // [rows, ld] fp32 or bf16
    long long ld;
    int rows, vocab;
    const int32_t *tokens;   // [rows] or null
    float factor;            // 1 / temperature
    int top;
    float *logprob, *entropy, *lse;   // [rows], each may be null
    int32_t *rank, *top_ids;
    float *top_logprobs;
};
cudaError_t launch_token_logprobs(const LogprobParams &p, bool bf16, cudaStream_t s);

struct LogprobGradParams {
    const void *logits;
    long long ld;
    int rows, vocab;
    const int32_t *tokens;   // [rows] or null
    float factor;
    const float *lse, *entropy, *grad_logprob, *grad_entropy;
    void *grad;
    long long ld_grad;
};
cudaError_t launch_token_logprobs_backward(const LogprobGradParams &p, bool bf16, cudaStream_t s);

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------

// The rows of a call that sequence b brings, clipped to [0, tokens) and max_tokens; what
// is clipped sets MTP_DEVERR_OFFSETS.
__device__ __forceinline__ void kv_rows(const KvParams &c, int b, int *first, int *count)
{
    if (c.starts == nullptr) {
        *count = c.tokens / c.batch;
        *first = b * *count;
        return;
    }
    const int lo = __ldg(c.starts + b), hi = __ldg(c.starts + b + 1);
    int n = hi - lo;
    if (lo < 0 || hi < lo || hi > c.tokens) n = 0;
    if (n > c.max_tokens) n = c.max_tokens;
    if (n != hi - lo && c.err) atomicOr(c.err, MTP_DEVERR_OFFSETS);
    *first = lo;
    *count = n;
}

__device__ __forceinline__ float bf16_value(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Code word -> value and value -> code of the two cache formats.
__device__ __forceinline__ float kv_value(uint8_t c, int format)
{
    if (format == MTP_KV_INT8) return (float)(int8_t)c;
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
    float f;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.f32.f16 %0, lo;\n}\n" : "=f"(f) : "r"(h2));
    return f;
}

__device__ __forceinline__ uint8_t kv_code(float v, int format)
{
    if (format == MTP_KV_INT8) return (uint8_t)(int8_t)__float2int_rn(fminf(fmaxf(v, -127.f), 127.f));
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return (uint8_t)r;
}

}  // namespace mtp
