/*
 * dq_serving.h — C ABI of the operators around the quantized products of
 * dq.h: the residual + root-mean-square norm that feeds an activation
 * quantizer, a paged key/value cache held in 4-bit codes, and attention over
 * that cache.
 *
 * Conventions are those of dq.h (device pointers, caller-owned buffers,
 * asynchronous calls ordered on `stream`, argument errors returned
 * synchronously with nothing launched, data errors raised as device flags
 * that dq_last_device_status() reports).  The codes and group scales are the
 * ones dq_quantize writes for the same rows with a = b = 1 and tensor scale 1.
 * (No counterpart in the method: the operators a quantized model is served
 * with.)
 */
#ifndef DQ_SERVING_H
#define DQ_SERVING_H

#include "dq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual addition, root-mean-square norm and activation quantization in one
 * pass:
 *     h[t, j]  = x[t, j] + residual[t, j]          (float32; residual may be NULL: h = x)
 *     residual_out[t, j] = bf16(h[t, j])           (NULL: not written)
 *     y[t, j]  = h[t, j] / sqrt(mean_j h[t, j]^2 + eps) * weight[j] * b[j]
 *     codes, gscales = Q(y)
 * The norm is taken of the unrounded h; y is formed and quantized in float32
 * (its codes are the exact rounding decisions on those float32 values).
 * x, residual: bf16, `tokens` rows of K elements, rows x_stride and
 * res_stride elements apart; residual_out: bf16, rows res_out_stride apart,
 * may be the same buffer as x or residual (same stride), and may not overlap
 * them otherwise (DQ_ERR_ARG; with another stride than theirs it lies outside
 * their extent).  weight: [K] of weight_dtype
 * (DQ_DT_F32 or DQ_DT_BF16); b: [K] float32, the inverse column scales of the
 * matrix that reads the result (dq_solve_dual_scale), or NULL for ones.
 * codes: dq_code_bytes(fmt, tokens, K) bytes; gscales [tokens, K/G]; every
 * format of dq.h.  K a multiple of G; strides at least K and multiples of 8
 * (16 bytes); x, residual, residual_out, codes, gscales, weight and b 16-byte
 * aligned; eps > 0.  A NaN or Inf in a row, or a sum of squares beyond
 * float32, raises DQ_ERR_NONFINITE; the codes of that row are then undefined.
 * No workspace. */
DQ_API dq_status dq_add_rmsnorm_quant(const void *x, int64_t x_stride, const void *residual,
                                      int64_t res_stride, const void *weight, int32_t weight_dtype,
                                      const float *b, float eps, int64_t tokens, int64_t K,
                                      const dq_format *fmt, void *residual_out,
                                      int64_t res_out_stride, uint8_t *codes, void *gscales,
                                      dq_stream stream);

/* A paged key/value cache.  Codes [pages, heads, page_size, head_dim / 2]
 * (two 4-bit codes per byte, the even channel low), group scales [pages,
 * heads, page_size, head_dim / G], for keys and values alike, in a format
 * with 4-bit codes (INT4 or E2M1).  head_dim 64 or 128, page_size a positive
 * multiple of 16; all four pointers 16-byte aligned. */
typedef struct dq_kv_cache {
    uint8_t *k_codes;
    void *k_scales;
    uint8_t *v_codes;
    void *v_scales;
    int64_t pages;
    int32_t page_size;
    int32_t heads;
    int32_t head_dim;
} dq_kv_cache;

/* A batch of sequences on that cache (device arrays, int32).  Sequence s has
 * kv_lens[s] tokens in all, of which the last new_s = starts[s+1] - starts[s]
 * are the new ones of this call: rows starts[s] .. starts[s+1] - 1 of the
 * call's token arrays, at positions kv_lens[s] - new_s ...  Position p lies
 * in page block_table[s * table_stride + p / page_size], slot p % page_size.
 * starts has seqs + 1 entries and does not decrease; new_s may be 0.  Rows
 * of the token arrays behind starts[seqs] belong to no sequence (padding):
 * they are neither read nor written.  Only the table entries of a sequence's
 * first ceil(kv_lens[s] / page_size) pages are read.
 * max_pages * page_size is at most 2^31 - 4096.
 * The contents are checked on the device: a sequence whose starts or length
 * lie out of range (starts decreasing or beyond `tokens`, kv_lens[s] < 0 or
 * beyond max_pages * page_size) is skipped, tokens whose position would be
 * negative or whose page is not in [0, pages) are not written (append), read
 * as zeros (read) or undefined for the rows that attend to them (attention);
 * each of these raises DQ_ERR_INDEX, and none leads to an access out of
 * bounds. */
typedef struct dq_kv_batch {
    const int32_t *starts;       /* [seqs + 1] */
    const int32_t *kv_lens;      /* [seqs] */
    const int32_t *block_table;  /* [seqs, table_stride], max_pages entries used per row */
    int32_t seqs;
    int32_t max_pages;
    int64_t table_stride;
} dq_kv_batch;

/* Quantize the new keys and values (bf16 [tokens, heads, head_dim]; the
 * channels contiguous, tokens and heads *_token and *_head elements apart,
 * strides multiples of 8) and write them to their places in the cache.  Every
 * (sequence, position) must have its own slot: two sequences that share a
 * page may only read it.  NaN or Inf raises DQ_ERR_NONFINITE.  No
 * workspace. */
DQ_API dq_status dq_kv_append(const void *k, int64_t k_token, int64_t k_head, const void *v,
                              int64_t v_token, int64_t v_head, int64_t tokens,
                              const dq_kv_cache *cache, const dq_kv_batch *batch,
                              const dq_format *fmt, dq_stream stream);

/* The values held in the cache for the batch's new tokens, code * group scale
 * rounded to bf16 (exact for E8M0 and E4M3 scales): the inverse of
 * dq_kv_append, with the same array layout (k and v may not overlap:
 * DQ_ERR_ARG; arrays of unequal strides lie outside each other's extent). */
DQ_API dq_status dq_kv_read(void *k, int64_t k_token, int64_t k_head, void *v, int64_t v_token,
                            int64_t v_head, int64_t tokens, const dq_kv_cache *cache,
                            const dq_kv_batch *batch, const dq_format *fmt, dq_stream stream);

/* Attention of the new tokens over the cache, which already holds them:
 *     out[t, h] = sum_p softmax_p(scale * q[t, h] . k[p, h / g]) v[p, h / g]
 * with g = q_heads / heads query heads per cache head and p over the
 * sequence's positions: all of them, or (causal != 0) those up to the token's
 * own.  A row that sees no position (an empty sequence, or more new tokens
 * than kv_lens with causal != 0) gives zeros.  q and out: bf16 [tokens,
 * q_heads, head_dim], channels contiguous, strides in elements, multiples of
 * 8; 16-byte aligned; `out` does not overlap q (DQ_ERR_ARG; with other strides
 * than q's it lies outside its extent).  Scores, softmax statistics
 * and sums are float32.  scale: finite, > 0.
 * Operands of the products are fp16, scaled by powers of two: queries per
 * row, what a product takes of values (and, above 32 query rows per sequence,
 * keys) per 32 positions, so that values 2^-24 below the largest group scale
 * of their 32 positions, or queries 2^-38 below their row's largest, count as
 * zero.  Keys may be up to 2^100 in magnitude (scores are formed with queries
 * scaled up to 2^14).  A query row with a NaN gives NaN; a NaN or infinite
 * group scale at a position of a sequence makes that sequence's rows of that
 * head undefined, and no others.
 * Workspace: dq_kv_attention_workspace bytes, 256-byte aligned, no
 * initialisation; calls that may overlap on the device need one each. */
DQ_API dq_status dq_kv_attention_workspace(int64_t tokens, int32_t q_heads, int32_t heads,
                                           int32_t head_dim, int32_t seqs, size_t *bytes);
DQ_API dq_status dq_kv_attention(const void *q, int64_t q_token, int64_t q_head, void *out,
                                 int64_t out_token, int64_t out_head, int64_t tokens,
                                 int32_t q_heads, float scale, int32_t causal,
                                 const dq_kv_cache *cache, const dq_kv_batch *batch,
                                 const dq_format *fmt, void *workspace, size_t ws_bytes,
                                 dq_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* DQ_SERVING_H */
