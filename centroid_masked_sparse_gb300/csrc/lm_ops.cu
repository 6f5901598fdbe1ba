// C ABI of the operators around the head: argument checks and launches.  Declarations and
// the contract of every entry point are in include/mtp_lm_ops.h.
#include <algorithm>
#include <cmath>

#include "lm_ops.h"

using namespace mtp;

namespace {

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

mtp_status cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return MTP_OK;
    cudaGetLastError();   // a failed call's error is not the next one's
    return MTP_ERR_CUDA;
}

mtp_status check_q4(int32_t rows, int32_t cols, int32_t group, int32_t device)
{
    if (rows < 1 || cols < 1 || device < 0) return MTP_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return MTP_ERR_UNSUPPORTED;
    if (cols % group != 0) return MTP_ERR_SHAPE;
    if (cols > MTP_Q4_MAX_COLS) return MTP_ERR_UNSUPPORTED;
    return MTP_OK;
}

mtp_status check_cache(const mtp_kv_desc *d, const mtp_kv_batch *s)
{
    if (!d || !s) return MTP_ERR_NULL;
    if (s->batch < 0 || s->tokens < 0 || d->device < 0) return MTP_ERR_SHAPE;
    if (d->num_pages < 1 || d->kv_heads < 1 || d->page_tokens < 16 || d->page_tokens % 16 != 0) return MTP_ERR_SHAPE;
    if (d->page_tokens > 1024 || d->kv_heads > 1024) return MTP_ERR_UNSUPPORTED;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return MTP_ERR_UNSUPPORTED;
    if (d->format != MTP_KV_INT8 && d->format != MTP_KV_E4M3) return MTP_ERR_UNSUPPORTED;
    if (s->batch == 0 || s->tokens == 0) return MTP_OK;
    if (!d->k_codes || !d->v_codes || !d->k_scales || !d->v_scales) return MTP_ERR_NULL;
    if (!s->page_table || !s->lengths) return MTP_ERR_NULL;
    if (s->batch > 65535) return MTP_ERR_UNSUPPORTED;
    if (s->max_tokens < 1 || s->table_width < 1 || s->ld_table < s->table_width) return MTP_ERR_SHAPE;
    if ((int64_t)s->table_width * d->page_tokens > 1 << 30) return MTP_ERR_UNSUPPORTED;
    if (!s->starts && s->tokens % s->batch != 0) return MTP_ERR_SHAPE;
    if (!aligned(d->k_codes, 16) || !aligned(d->v_codes, 16) || !aligned(d->k_scales, 4) || !aligned(d->v_scales, 4) ||
        !aligned(d->error_word, 4) || !aligned(s->page_table, 4) || !aligned(s->lengths, 4) || !aligned(s->starts, 4))
        return MTP_ERR_ALIGN;
    return MTP_OK;
}

mtp_status check_strides(const void *p, int64_t token, int64_t head)
{
    if (!p) return MTP_ERR_NULL;
    if (token < 0 || head < 0) return MTP_ERR_SHAPE;
    if (!aligned(p, 16) || token % 8 != 0 || head % 8 != 0) return MTP_ERR_ALIGN;
    return MTP_OK;
}

KvParams kv_params(const mtp_kv_desc *d, const mtp_kv_batch *s)
{
    KvParams c{};
    c.k_codes = (uint8_t *)d->k_codes;
    c.v_codes = (uint8_t *)d->v_codes;
    c.k_scales = d->k_scales;
    c.v_scales = d->v_scales;
    c.err = d->error_word;
    c.pages = d->num_pages;
    c.page_tokens = d->page_tokens;
    c.kv_heads = d->kv_heads;
    c.dim = d->head_dim;
    c.format = d->format;
    c.table = s->page_table;
    c.ld_table = s->ld_table;
    c.table_width = s->table_width;
    c.lengths = s->lengths;
    c.starts = s->starts;
    c.batch = s->batch;
    c.tokens = s->tokens;
    c.max_tokens = std::min(s->max_tokens, s->tokens);   // a bound of any size costs what the call's tokens do
    return c;
}

// Type, sizes and element alignment of rows of logits.
mtp_status check_logits(int32_t type, int64_t ld, int32_t rows, int32_t vocab, float temperature, int32_t device)
{
    if (type != MTP_TYPE_F32 && type != MTP_TYPE_BF16) return MTP_ERR_UNSUPPORTED;
    if (rows < 0 || vocab < 1 || ld < vocab || device < 0) return MTP_ERR_SHAPE;
    // the kernels multiply by log2(e) / temperature
    if (!(temperature > 0.f) || std::isinf(temperature) || std::isinf((float)(1.4426950408889634 / temperature))) return MTP_ERR_SHAPE;
    return MTP_OK;
}

}  // namespace

extern "C" {

size_t mtp_q4_packed_bytes(int32_t rows, int32_t cols, int32_t group, int32_t zeros)
{
    if (check_q4(rows, cols, group, 0) != MTP_OK) return 0;
    return q4_layout(rows, cols, group, zeros != 0).total;
}

mtp_status mtp_q4_pack(const mtp_q4_desc *d, const void *codes, int64_t ld_codes, const void *scales, const void *zeros,
                       void *packed, size_t packed_bytes, void *stream)
{
    if (!d) return MTP_ERR_NULL;
    mtp_status st = check_q4(d->rows, d->cols, d->group, d->device);
    if (st != MTP_OK) return st;
    if (!codes || !scales || (d->zeros != 0) != (zeros != nullptr) || !packed) return MTP_ERR_NULL;
    const Q4Layout L = q4_layout(d->rows, d->cols, d->group, d->zeros != 0);
    if (ld_codes < d->cols / 2 || packed_bytes < L.total) return MTP_ERR_SHAPE;
    if (!aligned(scales, 2) || !aligned(packed, 256)) return MTP_ERR_ALIGN;
    DeviceScope dev(d->device);
    if (!dev.ok) return MTP_ERR_CUDA;
    Q4PackParams p{};
    p.codes = (const uint8_t *)codes;
    p.ld_codes = ld_codes;
    p.scales = (const uint16_t *)scales;
    p.zeros = (const uint8_t *)zeros;
    p.M = d->rows;
    p.K = d->cols;
    p.G = d->cols / d->group;
    p.group = d->group;
    p.tiles = (int)(((int64_t)d->rows + 15) / 16);
    p.blocks = (d->cols + 63) / 64;
    p.out_codes = (uint8_t *)packed;
    p.out_scales = p.out_codes + L.scales;
    p.out_zeros = p.out_codes + L.zeros;
    return cuda_status(launch_q4_pack(p, (cudaStream_t)stream));
}

mtp_status mtp_q4_matvec(const mtp_q4_desc *d, const void *x, int64_t ld_x, int32_t batch, void *out, int32_t out_type,
                         int64_t ld_out, void *stream)
{
    if (!d) return MTP_ERR_NULL;
    mtp_status st = check_q4(d->rows, d->cols, d->group, d->device);
    if (st != MTP_OK) return st;
    if (out_type != MTP_TYPE_F32 && out_type != MTP_TYPE_BF16) return MTP_ERR_UNSUPPORTED;
    if (batch < 0 || !(d->softcap >= 0.f)) return MTP_ERR_SHAPE;
    if (batch > MTP_MAX_BATCH) return MTP_ERR_UNSUPPORTED;
    if (batch == 0) return MTP_OK;
    if (!d->packed || !x || !out) return MTP_ERR_NULL;
    if (ld_x < d->cols || ld_out < d->rows) return MTP_ERR_SHAPE;
    if (ld_x % 8 != 0 || !aligned(d->packed, 256) || !aligned(x, 16) || !aligned(out, out_type == MTP_TYPE_F32 ? 4 : 2))
        return MTP_ERR_ALIGN;
    DeviceScope dev(d->device);
    if (!dev.ok) return MTP_ERR_CUDA;
    const Q4Layout L = q4_layout(d->rows, d->cols, d->group, d->zeros != 0);
    Q4Params p{};
    p.codes = (const uint8_t *)d->packed;
    p.scales = p.codes + L.scales;
    p.zeros = d->zeros ? p.codes + L.zeros : nullptr;
    p.x = (const uint16_t *)x;
    p.ld_x = ld_x;
    p.out = out;
    p.ld_out = ld_out;
    p.M = d->rows;
    p.K = d->cols;
    p.group = d->group;
    p.blocks = (d->cols + 63) / 64;
    p.B = batch;
    p.bf16_out = out_type == MTP_TYPE_BF16;
    p.softcap = d->softcap;
    return cuda_status(launch_q4_matvec(p, (cudaStream_t)stream));
}

mtp_status mtp_q4_quantize(const void *w, int64_t ld_w, int32_t rows, int32_t cols, int32_t group, int32_t device,
                           void *codes, int64_t ld_codes, void *scales, void *zeros, void *stream)
{
    mtp_status st = check_q4(rows, cols, group, device);
    if (st != MTP_OK) return st;
    if (!w || !codes || !scales) return MTP_ERR_NULL;
    if (ld_w < cols || ld_codes < cols / 2) return MTP_ERR_SHAPE;
    if (!aligned(w, 2) || !aligned(scales, 2)) return MTP_ERR_ALIGN;
    DeviceScope dev(device);
    if (!dev.ok) return MTP_ERR_CUDA;
    return cuda_status(launch_q4_quantize((const uint16_t *)w, ld_w, rows, cols, group, (uint8_t *)codes, ld_codes,
                                          (uint16_t *)scales, (uint8_t *)zeros, (cudaStream_t)stream));
}

mtp_status mtp_kv_append(const mtp_kv_desc *d, const mtp_kv_batch *seqs, const void *k, int64_t k_token_stride,
                         int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                         void *stream)
{
    mtp_status st = check_cache(d, seqs);
    if (st != MTP_OK || seqs->batch == 0 || seqs->tokens == 0) return st;
    if ((st = check_strides(k, k_token_stride, k_head_stride)) != MTP_OK) return st;
    if ((st = check_strides(v, v_token_stride, v_head_stride)) != MTP_OK) return st;
    DeviceScope dev(d->device);
    if (!dev.ok) return MTP_ERR_CUDA;
    KvAppendParams p{};
    p.c = kv_params(d, seqs);
    p.k = (const uint16_t *)k;
    p.v = (const uint16_t *)v;
    p.k_token = k_token_stride;
    p.k_head = k_head_stride;
    p.v_token = v_token_stride;
    p.v_head = v_head_stride;
    return cuda_status(launch_kv_append(p, (cudaStream_t)stream));
}

size_t mtp_kv_attention_workspace_bytes(const mtp_kv_desc *d, const mtp_kv_batch *seqs, int32_t heads, int32_t max_len,
                                        int32_t window)
{
    if (check_cache(d, seqs) != MTP_OK || heads < 1 || heads % d->kv_heads != 0 || max_len < 0 || window < 0) return 0;
    if (seqs->batch == 0 || seqs->tokens == 0) return MTP_KV_WORKSPACE_ZEROED;
    DeviceScope dev(d->device);   // the split depends on the device's SMs
    if (!dev.ok && dev.prev >= 0) return 0;   // no such device (without any GPU: sizes as for one SM)
    return MTP_KV_WORKSPACE_ZEROED + kv_attention_plan(kv_params(d, seqs), heads, window, max_len).partial_floats * sizeof(float);
}

mtp_status mtp_kv_attention(const mtp_kv_desc *d, const mtp_kv_batch *seqs, const void *q, int64_t q_token_stride,
                            int64_t q_head_stride, int32_t heads, int32_t max_len, int32_t window, float scale,
                            void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    mtp_status st = check_cache(d, seqs);
    if (st != MTP_OK) return st;
    if (heads < 1 || heads % d->kv_heads != 0 || max_len < 0 || window < 0) return MTP_ERR_SHAPE;
    if (heads > 65535) return MTP_ERR_UNSUPPORTED;
    if (seqs->batch == 0 || seqs->tokens == 0) return MTP_OK;
    if ((int64_t)(seqs->starts ? std::min(seqs->max_tokens, seqs->tokens) : seqs->tokens / seqs->batch) * heads > 1 << 19)
        return MTP_ERR_UNSUPPORTED;
    if ((st = check_strides(q, q_token_stride, q_head_stride)) != MTP_OK) return st;
    if (!out) return MTP_ERR_NULL;
    if (!workspace || workspace_bytes < MTP_KV_WORKSPACE_ZEROED) return MTP_ERR_WORKSPACE;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16)) return MTP_ERR_ALIGN;
    DeviceScope dev(d->device);
    if (!dev.ok) return MTP_ERR_CUDA;
    KvAttentionParams p{};
    p.c = kv_params(d, seqs);
    const KvAttentionPlan plan = kv_attention_plan(p.c, heads, window, max_len);
    if (workspace_bytes < MTP_KV_WORKSPACE_ZEROED + plan.partial_floats * sizeof(float)) return MTP_ERR_WORKSPACE;
    p.tickets = (uint32_t *)workspace;
    p.partial = (float *)((char *)workspace + MTP_KV_WORKSPACE_ZEROED);
    p.q = (const uint16_t *)q;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.heads = heads;
    p.window = window;
    p.scale = scale;
    p.out = (uint16_t *)out;
    p.lse = lse;
    return cuda_status(launch_kv_attention(p, plan, (cudaStream_t)stream));
}

mtp_status mtp_token_logprobs(const void *logits, int32_t type, int64_t ld, int32_t rows, int32_t vocab,
                              const int32_t *tokens, float temperature, int32_t top, float *logprob, float *entropy,
                              int32_t *rank, float *lse, int32_t *top_ids, float *top_logprobs, int32_t device,
                              void *stream)
{
    mtp_status st = check_logits(type, ld, rows, vocab, temperature, device);
    if (st != MTP_OK) return st;
    if (top < 0) return MTP_ERR_SHAPE;
    if (top > MTP_MAX_TOP) return MTP_ERR_UNSUPPORTED;
    if (rows == 0) return MTP_OK;
    if (!logits || (!tokens && (logprob || rank)) || (top > 0 && !top_ids)) return MTP_ERR_NULL;
    if (!aligned(logits, type == MTP_TYPE_F32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logprob, 4) ||
        !aligned(entropy, 4) || !aligned(rank, 4) || !aligned(lse, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
        return MTP_ERR_ALIGN;
    DeviceScope dev(device);
    if (!dev.ok) return MTP_ERR_CUDA;
    LogprobParams p{};
    p.logits = logits;
    p.ld = ld;
    p.rows = rows;
    p.vocab = vocab;
    p.tokens = tokens;
    p.factor = (float)(1.0 / temperature);
    p.top = top;
    p.logprob = logprob;
    p.entropy = entropy;
    p.lse = lse;
    p.rank = rank;
    p.top_ids = top_ids;
    p.top_logprobs = top_logprobs;
    return cuda_status(launch_token_logprobs(p, type == MTP_TYPE_BF16, (cudaStream_t)stream));
}

mtp_status mtp_token_logprobs_backward(const void *logits, int32_t type, int64_t ld, int32_t rows, int32_t vocab,
                                       const int32_t *tokens, float temperature, const float *lse, const float *entropy,
                                       const float *grad_logprob, const float *grad_entropy, void *grad_logits,
                                       int64_t ld_grad, int32_t device, void *stream)
{
    mtp_status st = check_logits(type, ld, rows, vocab, temperature, device);
    if (st != MTP_OK) return st;
    if (ld_grad < vocab) return MTP_ERR_SHAPE;
    if (rows == 0) return MTP_OK;
    if (!logits || !lse || !grad_logits || (!grad_logprob && !grad_entropy) || (grad_logprob && !tokens) ||
        (grad_entropy && !entropy))
        return MTP_ERR_NULL;
    if (logits == grad_logits && ld != ld_grad) return MTP_ERR_SHAPE;
    const size_t size = type == MTP_TYPE_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(grad_logits, size) || !aligned(tokens, 4) || !aligned(lse, 4) ||
        !aligned(entropy, 4) || !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4))
        return MTP_ERR_ALIGN;
    DeviceScope dev(device);
    if (!dev.ok) return MTP_ERR_CUDA;
    LogprobGradParams p{};
    p.logits = logits;
    p.ld = ld;
    p.rows = rows;
    p.vocab = vocab;
    p.tokens = tokens;
    p.factor = (float)(1.0 / temperature);
    p.lse = lse;
    p.entropy = entropy;
    p.grad_logprob = grad_logprob;
    p.grad_entropy = grad_entropy;
    p.grad = grad_logits;
    p.ld_grad = ld_grad;
    return cuda_status(launch_token_logprobs_backward(p, type == MTP_TYPE_BF16, (cudaStream_t)stream));
}

}  // extern "C"
