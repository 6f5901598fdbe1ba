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
    int M, K, group, B;
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
    uint32_t *tickets;       // [items][8], zero between calls
    float *partial;          // sums of the clusters of an item
    int row_tiles, splits;   // set by the plan
    uint32_t page_magic;     // block / (page_tokens / 16) = umulhi(block, magic), 0: no division
};
// How a call is split: CTAs per item (a sequence, a kv head and a tile of query rows), in
// clusters of `cluster`; the floats that the items' clusters exchange.
struct KvAttentionPlan {
    int tiles8;              // query rows of an item / 8 (1 or 2)
    int row_tiles, splits, cluster;
    long long items;
    size_t partial_floats;
};
KvAttentionPlan kv_attention_plan(const KvParams &c, int heads, int window, int max_len);
cudaError_t launch_kv_attention(KvAttentionParams p, const KvAttentionPlan &plan, cudaStream_t s);

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

// Launch in clusters of `cluster` CTAs along x, behind the kernel ahead of it on the stream as
// launch_dependent does.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------

// The rows of a call that sequence b brings, clipped to [0, tokens) and max_tokens; what
// is clipped sets MTP_DEVERR_OFFSETS.  Returns how many it brings with those beyond max_tokens.
__device__ __forceinline__ int kv_rows(const KvParams &c, int b, int *first, int *count)
{
    if (c.starts == nullptr) {
        *count = c.tokens / c.batch;
        *first = b * *count;
        return *count;
    }
    const int lo = __ldg(c.starts + b), hi = __ldg(c.starts + b + 1);
    const bool good = lo >= 0 && hi >= lo && hi <= c.tokens;
    const int all = good ? hi - lo : 0;
    *first = lo;
    *count = min(all, c.max_tokens);
    if ((!good || *count != all) && c.err) atomicOr(c.err, MTP_DEVERR_OFFSETS);
    return all;
}

__device__ __forceinline__ float bf16_value(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// A code's value in the two cache formats.
__device__ __forceinline__ float kv_value(uint32_t c, int format)
{
    if (format == MTP_KV_INT8) return (float)(int8_t)c;
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(c & 255u)));
    float f;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.f32.f16 %0, lo;\n}\n" : "=f"(f) : "r"(h2));
    return f;
}

// Four values -> four codes, the first in the low byte.
__device__ __forceinline__ uint32_t kv_codes(float a, float b, float c, float d, int format)
{
    if (format == MTP_KV_INT8) {
        auto code = [](float v) { return (uint32_t)__float2int_rn(fminf(fmaxf(v, -127.f), 127.f)) & 255u; };
        return code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
    }
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        " mov.b32 %0, {lo, hi};\n}\n" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// 16 bytes from global to shared memory without a register or L1.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// d += a * b of m16n8k16, fp16 in, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// acc += s * d on a pair, with one instruction.
__device__ __forceinline__ void fma_pair(float &acc0, float &acc1, float s, float d0, float d1)
{
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%0, %1};\n"
        " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}\n"
        : "+f"(acc0), "+f"(acc1)
        : "f"(d0), "f"(d1), "f"(s));
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The first `bytes` (0 or 16) of 16; the rest of the destination is zeroed.
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8_part(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// d = a * b + c with c[0] = c[2], c[1] = c[3] (the same for every row).
__device__ __forceinline__ void mma_f16_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1, float c0, float c1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// Transpose of an 8 x 8 matrix of 16-bit values, one row per quad of lanes.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The power of two that brings the bf16 value with these bits (no sign) to [2^14, 2^15),
// as its exponent field, and its inverse.
__device__ __forceinline__ uint32_t fp16_factor_field(uint32_t top) { return top == 0 ? 127u : min(254u, 268u - (top >> 7)); }
__device__ __forceinline__ float fp16_factor_inverse(uint32_t e) { return __uint_as_float(e == 254u ? 0x00400000u : (254u - e) << 23); }

// Every kernel here starts with the first: it may be brought up while the one ahead of it on
// the stream ends, and touches no memory before that one is through.  The second lets the next
// kernel be brought up before this one ends; only with one CTA per SM, where the next one's
// cannot take the places of CTAs to come (with several it gains nothing: attention over 65519
// tokens 18.2 us in a graph, without 18.1, over 64 ragged sequences 128.4 and 128.0).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Thread-block clusters.
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Its halves without an order of memory: no CTA is past the second before all are past the first.
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// A float of another CTA's shared memory: the address of one's own copy, and the rank.
__device__ __forceinline__ float cluster_load(const float *own, uint32_t rank)
{
    const uint32_t addr = (uint32_t)__cvta_generic_to_shared(own);
    float v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}\n"
                 : "=f"(v) : "r"(addr), "r"(rank) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_load4(const float *own, uint32_t rank)
{
    const uint32_t addr = (uint32_t)__cvta_generic_to_shared(own);
    float4 v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank) : "memory");
    return v;
}

}  // namespace mtp
