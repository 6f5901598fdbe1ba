/*
 * mtp_lm_ops.h - C ABI of the operators around the masked head, for GB300 (sm_103a).
 *
 * What a draft model and its verifier run next to the head of mtp_head.h:
 *   mtp_q4_matvec          products with a 4-bit weight matrix (a projection of the
 *                          draft model, or the target's head over every vocabulary row)
 *   mtp_kv_append          new keys and values into a paged cache held in 8 bits
 *   mtp_kv_attention       attention of one or a few query tokens per sequence over it
 *   mtp_token_logprobs     log probability of a given token per row of logits, its rank,
 *                          the row's entropy and its largest alternatives
 *   mtp_token_logprobs_backward   the gradient of those log probabilities and entropies
 *
 * The conventions of mtp_head.h hold: caller-owned device pointers on one device, no
 * allocation, no synchronisation, no device memory read on the host, launches on
 * `stream` only; host-side checks run before anything is launched; the calling thread
 * keeps its current device.  Calls on an empty batch (rows, tokens or batch 0) return
 * MTP_OK and launch nothing.
 */
#ifndef MTP_LM_OPS_H
#define MTP_LM_OPS_H

#include "mtp_head.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of logits, gradients and products. */
#define MTP_TYPE_F32 0
#define MTP_TYPE_BF16 1

/* ---------------------------------------------------------------------------
 * 4-bit weights
 * ------------------------------------------------------------------------ */

/* A matrix of `rows` x `cols` weights in 4 bits, with one scale (and optionally one
 * zero point) for each group of `group` consecutive columns of a row:
 *   w[m, k] = (code[m, k] - z) * scale[m, k / group],   z = zero[m, k / group] or 8.
 *   rows      M >= 1
 *   cols      K, a multiple of group, 32 <= K <= MTP_Q4_MAX_COLS
 *   group     32, 64 or 128
 *   zeros     whether there are zero points (0: 8 everywhere)
 *   device    CUDA ordinal of every buffer
 *   packed    the matrix as mtp_q4_pack lays it out, 256-byte aligned
 *   softcap   each product y becomes cap * tanh(y / cap); 0: none; negative or NaN:
 *             MTP_ERR_SHAPE */
#define MTP_Q4_MAX_COLS 16384
typedef struct mtp_q4_desc {
    int32_t rows;
    int32_t cols;
    int32_t group;
    int32_t zeros;
    int32_t device;
    const void *packed;
    float softcap;
} mtp_q4_desc;

/* The packed matrix: mtp_q4_pack lays codes, scales and zero points out once, like loading
 * the weights, in the order in which mtp_q4_matvec's warps read them; what it was packed
 * from need not be kept.  Rows go in tiles of 16, columns in blocks of 64 (codes) and steps
 * of 256 (scales), with T = ceil(M / 16), B = ceil(K / 64), S = ceil(K / 256),
 * n = 256 / group, and each part padded to 256 bytes:
 *   codes    uint32 [T][B][32 lanes][4]: of lane 4g + t, word j holds row g + (j % 2) * 8 of
 *            the tile and columns 64 b + (j / 2) * 32 + 8t .. + 7, the lowest four bits first
 *   scales   bf16 [T][S][8][n][2]: of row g (then g + 8) and group s * n + i
 *   zeros    uint8 of the same shape (only if there are any)
 * with zeros in place of what the matrix does not have.  mtp_q4_packed_bytes: the size, or
 * 0 for invalid sizes.
 *   codes     uint8 [M, ld_codes]: byte j of a row holds column 2j in its low and
 *             column 2j + 1 in its high four bits; ld_codes >= K / 2 bytes
 *   scales    bf16 [M, K / group] contiguous
 *   zeros     uint8 [M, K / group] contiguous (only the low four bits are read); not NULL
 *             exactly if desc->zeros
 * desc->packed and softcap are not read. */
MTP_API size_t mtp_q4_packed_bytes(int32_t rows, int32_t cols, int32_t group, int32_t zeros);
MTP_API mtp_status mtp_q4_pack(const mtp_q4_desc *desc, const void *codes, int64_t ld_codes, const void *scales,
                               const void *zeros, void *packed, size_t packed_bytes, void *stream);

/* out[b, m] = softcap(sum_k w[m, k] * x[b, k]).
 *   x         bf16 [batch, ld_x], 16-byte aligned, ld_x >= K and a multiple of 8
 *   out       [batch, ld_out] of out_type (MTP_TYPE_F32, or MTP_TYPE_BF16: rounded once,
 *             to nearest even), aligned to its element, ld_out >= M
 *   batch     0..MTP_MAX_BATCH; each 32 rows read the codes once
 * Codes and zero points enter the products exactly, x to 2^-35 of its row's largest value
 * or better (all of its 8 bits, unless it is below 2^-25 of that); sums, scales and the
 * softcap are fp32.  A row of x that holds a NaN or an infinity gives NaN; non-finite scales
 * give what IEEE arithmetic gives in their outputs only. */
MTP_API mtp_status mtp_q4_matvec(const mtp_q4_desc *desc, const void *x, int64_t ld_x, int32_t batch,
                                 void *out, int32_t out_type, int64_t ld_out, void *stream);

/* Round a bf16 matrix w [rows, ld_w] (finite values) to codes, scales and zero points in
 * the layout that mtp_q4_pack reads; a one-time step.  Per group, in fp32 with IEEE division:
 *   zeros == NULL   scale = bf16(max|w| / 7), code = clamp(rint(w / scale) + 8, 0, 15)
 *   otherwise       lo = min(0, min w), hi = max(0, max w), scale = bf16((hi - lo) / 15),
 *                   zero = clamp(rint(-lo / scale), 0, 15),
 *                   code = clamp(rint(w / scale) + zero, 0, 15)
 * (scale 0: the code is the zero point, 8 or 0).  ld_codes >= cols / 2, any value. */
MTP_API mtp_status mtp_q4_quantize(const void *w, int64_t ld_w, int32_t rows, int32_t cols, int32_t group,
                                   int32_t device, void *codes, int64_t ld_codes, void *scales, void *zeros,
                                   void *stream);

/* ---------------------------------------------------------------------------
 * The 8-bit cache
 * ------------------------------------------------------------------------ */

#define MTP_KV_INT8 0 /* signed integers -127..127                    */
#define MTP_KV_E4M3 1 /* 8-bit floats, 4 exponent and 3 mantissa bits */

/* Device error bits of these calls (OR-ed into desc->error_word, never cleared here):
 *   MTP_DEVERR_PAGE     a page id outside [0, num_pages) or a length beyond the table:
 *                       its tokens are skipped (not written, not attended to)
 *   MTP_DEVERR_OFFSETS  starts not ascending inside [0, tokens], or more tokens in a
 *                       sequence than max_tokens: the tokens beyond are skipped (their
 *                       outputs are not written), the others keep their places */
#define MTP_DEVERR_PAGE 0x8u

/* A paged cache of keys and values.  A page holds page_tokens consecutive tokens of one
 * sequence for every kv head; the page is the block that shares a scale per head:
 *   key of token p of head h = k_codes[page, h, p % page_tokens, :] * k_scales[page, h]
 *   num_pages     >= 1
 *   page_tokens   a multiple of 16, 16..1024
 *   kv_heads      1..1024
 *   head_dim      64, 128 or 256
 *   format        MTP_KV_INT8 or MTP_KV_E4M3
 *   k_codes,      uint8 [num_pages, kv_heads, page_tokens, head_dim] contiguous, 16-byte
 *   v_codes       aligned
 *   k_scales,     fp32 [num_pages, kv_heads]
 *   v_scales
 *   error_word    device uint32, or NULL (errors are then only skipped) */
typedef struct mtp_kv_desc {
    int32_t num_pages;
    int32_t page_tokens;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t format;
    int32_t device;
    void *k_codes;
    void *v_codes;
    float *k_scales;
    float *v_scales;
    uint32_t *error_word;
} mtp_kv_desc;

/* The sequences of a call and the tokens that each brings.
 *   batch        sequences, 0..65535
 *   tokens       tokens of the call in all (rows of k, v or q)
 *   max_tokens   the most tokens that one sequence brings (a bound, >= 1; above `tokens` it
 *                counts as `tokens`)
 *   table_width  page ids per sequence in the table, >= 1, table_width * page_tokens <= 2^30
 *   page_table   int32 [batch, ld_table]: page of a sequence's tokens
 *                [i * page_tokens, (i + 1) * page_tokens) at column i; columns that no
 *                token of the call or of the sequence needs are not read
 *   ld_table     elements between its rows, >= table_width
 *   lengths      int32 [batch]: mtp_kv_append: the tokens already in the cache;
 *                mtp_kv_attention: the tokens in the cache, the call's own included
 *   starts       int32 [batch + 1]: sequence b brings rows [starts[b], starts[b + 1]);
 *                NULL: tokens / batch rows each (MTP_ERR_SHAPE if that leaves a rest) */
typedef struct mtp_kv_batch {
    int32_t batch;
    int32_t tokens;
    int32_t max_tokens;
    int32_t table_width;
    const int32_t *page_table;
    int64_t ld_table;
    const int32_t *lengths;
    const int32_t *starts;
} mtp_kv_batch;

/* Write the call's tokens behind each sequence's own.  For each block that they reach,
 * per head and separately for keys and values, in fp32 with IEEE division:
 *   scale' = max(scale if the block holds earlier tokens of the sequence else 0,
 *                max|x_new| / Q),   Q = 127 (int8) or 448 (e4m3)
 *   earlier codes c become round(c * (scale / scale')), new ones round(x / scale')
 * (to nearest even; scale' = 0: codes 0).  Codes behind the last token stay as they are.
 * NaN counts as 0 and infinities as the largest finite bf16.
 *   k, v   bf16 [tokens, kv_heads, head_dim] with unit stride inside a head and the given
 *          strides, in elements (multiples of 8), between tokens and heads; 16-byte aligned
 * Sequences of one call must not share the blocks that they write. */
MTP_API mtp_status mtp_kv_append(const mtp_kv_desc *desc, const mtp_kv_batch *seqs, const void *k,
                                 int64_t k_token_stride, int64_t k_head_stride, const void *v,
                                 int64_t v_token_stride, int64_t v_head_stride, void *stream);

/* Attention of each sequence's query tokens over its cached tokens.  Query i of n in a
 * sequence of L tokens stands at position p = L - n + i and sees positions
 * max(0, p - window + 1) .. p (window 0: from 0).  Query head j reads kv head
 * j / (heads / kv_heads).  Per query token and head:
 *   o = sum_j e^(s_j - lse) v_j,   s_j = scale * (q . k_j),   lse = ln sum_j e^(s_j)
 * A query that sees nothing (p < 0) gets o = 0 and lse = -inf.
 *   q        bf16 [tokens, heads, head_dim], strides as for mtp_kv_append
 *   heads    a multiple of kv_heads, max_tokens * heads <= 2^19 (without starts: tokens / batch * heads)
 *   max_len  a bound on the lengths that decides how the work is split (any length is
 *            right); 0: table_width * page_tokens
 *   out      bf16 [tokens, heads, head_dim] contiguous, 16-byte aligned
 *   lse      fp32 [tokens, heads] contiguous, or NULL
 *   workspace  mtp_kv_attention_workspace_bytes bytes, 16-byte aligned, whose first
 *              MTP_KV_WORKSPACE_ZEROED bytes are zero before the first call that uses it;
 *              calls leave them zero.  One call at a time, like every workspace.  Its size is 0
 *              for arguments or a device that the call would refuse.
 * Scores, softmax statistics and sums are fp32; keys, values and q enter the products
 * exactly, and the weights e^(s_j - max) of the value sums with 11 significant bits, those
 * below 2^-21 to 2^-32.
 * Non-finite q, scales or e4m3 codes give what IEEE arithmetic gives (an infinite scale of
 * values that not every query of a sequence sees: NaN), in the queries that see them only. */
#define MTP_KV_WORKSPACE_ZEROED 262144u
MTP_API size_t mtp_kv_attention_workspace_bytes(const mtp_kv_desc *desc, const mtp_kv_batch *seqs, int32_t heads,
                                                int32_t max_len, int32_t window);
MTP_API mtp_status mtp_kv_attention(const mtp_kv_desc *desc, const mtp_kv_batch *seqs, const void *q,
                                    int64_t q_token_stride, int64_t q_head_stride, int32_t heads, int32_t max_len,
                                    int32_t window, float scale, void *out, float *lse, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Token log probabilities
 * ------------------------------------------------------------------------ */

#define MTP_MAX_TOP 32

/* For each row of logits, with x = logits / temperature and p = softmax(x):
 *   logprob[r]   ln p[token[r]]; 0 for a row without a given token
 *   rank[r]      how many tokens come before the given one, by (logit desc, id asc); -1
 *                for a row without a given token
 *   entropy[r]   -sum p ln p
 *   lse[r]       ln sum e^x
 *   top_ids[r, i], top_logprobs[r, i]   the i-th largest logit's token id and ln p, by
 *                (logit desc, id asc); -1 and -inf beyond the row's logits above -inf
 * Logits / temperature have to stay within fp32's range.
 * Logits of -inf are masked tokens: they have p = 0, and a row of nothing else gives
 * lse = -inf, logprob = -inf and entropy 0.  A NaN or +inf makes the row's logprob,
 * entropy, lse and top_logprobs NaN; its rank and top_ids are then unspecified.
 *   logits       [rows, ld] of type (MTP_TYPE_*), aligned to its element, ld >= vocab
 *   tokens       int32 [rows], an id outside [0, vocab) marking a row without one; NULL
 *                if logprob and rank are NULL
 *   temperature  > 0 and finite, as log2(e) / temperature (4.3e-39 and up)
 *   top          0..MTP_MAX_TOP alternatives (top_ids and top_logprobs [rows, top])
 * Every output may be NULL; NULL top_ids with top > 0 gives MTP_ERR_NULL. */
MTP_API mtp_status mtp_token_logprobs(const void *logits, int32_t type, int64_t ld, int32_t rows, int32_t vocab,
                                      const int32_t *tokens, float temperature, int32_t top, float *logprob,
                                      float *entropy, int32_t *rank, float *lse, int32_t *top_ids,
                                      float *top_logprobs, int32_t device, void *stream);

/* The gradient of sum_r grad_logprob[r] * logprob[r] + grad_entropy[r] * entropy[r]:
 *   grad_logits[r, i] = (g_l * ((i == token) - p_i) - g_e * p_i * (ln p_i + entropy[r])) / temperature
 * with g_l taken as 0 for a row without a given token; masked tokens get 0.
 *   lse, entropy   of the forward call (entropy is read only with grad_entropy).  p has a
 *                relative error of up to 2^-22 |lse| from lse's own roundings; a row of |lse| >=
 *                1024 is summed again instead.  A p below 2^-126 counts as 0
 *   grad_logprob, grad_entropy   fp32 [rows]; either may be NULL, not both; tokens may be
 *                NULL without grad_logprob
 *   grad_logits  [rows, ld_grad] of the logits' type; may be the logits themselves (same
 *                address and ld), otherwise must not overlap them */
MTP_API mtp_status mtp_token_logprobs_backward(const void *logits, int32_t type, int64_t ld, int32_t rows,
                                               int32_t vocab, const int32_t *tokens, float temperature,
                                               const float *lse, const float *entropy, const float *grad_logprob,
                                               const float *grad_entropy, void *grad_logits, int64_t ld_grad,
                                               int32_t device, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MTP_LM_OPS_H */
