// dq_serving_api.cu — the C ABI of include/dq_serving.h: argument checks and
// launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "dq_serving.h"

using namespace dq;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

dq_status launched(cudaError_t e, int n) {
    if (e != cudaSuccess) return DQ_ERR_CUDA;
    serving_count_launches(n);
    return DQ_OK;
}

// The format, cache and batch of a call (and its number of token rows).
dq_status check_cache(const dq_kv_cache *c, const dq_kv_batch *b, const dq_format *fmt, int64_t tokens) {
    if (!c || !b) return DQ_ERR_ARG;
    int bits = 0;
    const dq_status s = serving_format(fmt, &bits);
    if (s != DQ_OK) return s;
    if (bits != 4) return DQ_ERR_FORMAT;
    if (c->head_dim != 64 && c->head_dim != 128) return DQ_ERR_SHAPE;
    if (c->page_size <= 0 || c->page_size % 16 || c->heads <= 0 || c->pages < 0) return DQ_ERR_SHAPE;
    if (c->heads > 65535 || c->pages > INT32_MAX) return DQ_ERR_SHAPE;
    if (b->seqs < 0 || b->max_pages < 0 || b->table_stride < b->max_pages) return DQ_ERR_SHAPE;
    // (the kernels look up to 4095 positions past a sequence's end in 32 bits)
    if ((int64_t)b->max_pages * c->page_size > INT32_MAX - 4095) return DQ_ERR_SHAPE;
    if (tokens < 0 || tokens > INT32_MAX) return DQ_ERR_SHAPE;
    if (tokens == 0 || b->seqs == 0) return DQ_OK;
    if (!b->starts || !b->kv_lens) return DQ_ERR_ARG;
    if (b->max_pages > 0 && !b->block_table) return DQ_ERR_ARG;
    if (c->pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)) return DQ_ERR_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
        !aligned(c->v_scales, 16) || !aligned(b->starts, 4) || !aligned(b->kv_lens, 4) ||
        !aligned(b->block_table, 4))
        return DQ_ERR_ALIGN;
    return DQ_OK;
}

// Whether two bf16 arrays [tokens, heads, dim] share an element.  Exact where
// both have the same strides (interleaved slices of one array do not overlap);
// otherwise whether their extents meet.
bool overlap(const void *pa, int64_t token_a, int64_t head_a, const void *pb, int64_t token_b,
             int64_t head_b, int64_t tokens, int64_t heads, int64_t dim) {
    if (!pa || !pb) return false;
    const auto extent = [&](int64_t token, int64_t head) { return (tokens - 1) * token + (heads - 1) * head + dim; };
    const int64_t d = ((intptr_t)pb - (intptr_t)pa) / 2;       // (both are 16-byte aligned)
    if (d >= extent(token_a, head_a) || -d >= extent(token_b, head_b)) return false;
    if ((tokens > 1 && token_a != token_b) || (heads > 1 && head_a != head_b)) return true;
    // rows i tokens and j heads apart, for each j the i that bring them closest
    for (int64_t j = 1 - heads; j < heads; ++j) {
        const int64_t x = d + j * head_a, near = token_a ? -x / token_a : 0;
        for (int64_t i = near - 1; i <= near + 1; ++i) {
            const int64_t y = x + std::min(std::max(i, 1 - tokens), tokens - 1) * token_a;
            if (y < dim && -y < dim) return true;
        }
    }
    return false;
}

// A bf16 array [tokens, heads, dim] by its strides (16-byte accesses); an
// array that is written may not overlap itself.
dq_status check_rows(const void *p, int64_t token, int64_t head, int64_t tokens, int64_t heads,
                     int64_t dim, bool written) {
    if (!p) return DQ_ERR_ARG;
    if (token < 0 || head < 0 || token % 8 || head % 8) return DQ_ERR_SHAPE;
    if (written && !(token >= (heads - 1) * head + dim && (heads == 1 || head >= dim)) &&
        !(head >= (tokens - 1) * token + dim && (tokens == 1 || token >= dim)))
        return DQ_ERR_SHAPE;
    if (!aligned(p, 16)) return DQ_ERR_ALIGN;
    return DQ_OK;
}

dq_status kv_copy(const void *k, int64_t k_token, int64_t k_head, const void *v, int64_t v_token,
                  int64_t v_head, int64_t tokens, const dq_kv_cache *cache, const dq_kv_batch *batch,
                  const dq_format *fmt, dq_stream stream, bool read) {
    dq_status s = check_cache(cache, batch, fmt, tokens);
    if (s != DQ_OK) return s;
    if (tokens == 0 || batch->seqs == 0) return DQ_OK;
    if ((s = check_rows(k, k_token, k_head, tokens, cache->heads, cache->head_dim, read)) != DQ_OK) return s;
    if ((s = check_rows(v, v_token, v_head, tokens, cache->heads, cache->head_dim, read)) != DQ_OK) return s;
    if (read && overlap(k, k_token, k_head, v, v_token, v_head, tokens, cache->heads, cache->head_dim))
        return DQ_ERR_ARG;
    KvCopyLaunch L;
    L.status = serving_status_word();
    if (!L.status) return DQ_ERR_CUDA;
    L.k = k;
    L.v = v;
    L.k_token = k_token;
    L.k_head = k_head;
    L.v_token = v_token;
    L.v_head = v_head;
    L.tokens = tokens;
    L.cache = *cache;
    L.batch = *batch;
    L.codes = fmt->codes;
    L.gscale = fmt->group_scale;
    L.group = fmt->group;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(read ? launch_kv_read(L) : launch_kv_append(L), 1);
}

}  // namespace

extern "C" {

dq_status dq_add_rmsnorm_quant(const void *x, int64_t x_stride, const void *residual,
                               int64_t res_stride, const void *weight, int32_t weight_dtype,
                               const float *b, float eps, int64_t tokens, int64_t K,
                               const dq_format *fmt, void *residual_out, int64_t res_out_stride,
                               uint8_t *codes, void *gscales, dq_stream stream) {
    const dq_status s = serving_format(fmt, nullptr);
    if (s != DQ_OK) return s;
    if (weight_dtype != DQ_DT_F32 && weight_dtype != DQ_DT_BF16) return DQ_ERR_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return DQ_ERR_ARG;
    if (tokens < 0 || tokens > INT32_MAX || K < 0 || K > (1 << 28) || K % fmt->group) return DQ_ERR_SHAPE;
    if (tokens == 0 || K == 0) return DQ_OK;
    if (!x || !weight || !codes || !gscales) return DQ_ERR_ARG;
    if (x_stride < K || x_stride % 8) return DQ_ERR_SHAPE;
    if (residual && (res_stride < K || res_stride % 8)) return DQ_ERR_SHAPE;
    if (residual_out && (res_out_stride < K || res_out_stride % 8)) return DQ_ERR_SHAPE;
    if (residual_out && residual_out == residual && res_out_stride != res_stride) return DQ_ERR_SHAPE;
    if (residual_out && residual_out == x && res_out_stride != x_stride) return DQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(b, 16) ||
        !aligned(residual_out, 16) || !aligned(codes, 16) || !aligned(gscales, 16))
        return DQ_ERR_ALIGN;
    // (in place: a row's elements are read before they are written)
    if (residual_out != x && overlap(x, x_stride, 0, residual_out, res_out_stride, 0, tokens, 1, K)) return DQ_ERR_ARG;
    if (residual_out != residual && overlap(residual, res_stride, 0, residual_out, res_out_stride, 0, tokens, 1, K))
        return DQ_ERR_ARG;
    NormLaunch L;
    L.status = serving_status_word();
    if (!L.status) return DQ_ERR_CUDA;
    L.x = x;
    L.residual = residual;
    L.x_stride = x_stride;
    L.res_stride = res_stride;
    L.weight = weight;
    L.weight_f32 = weight_dtype == DQ_DT_F32;
    L.b = b;
    L.eps = eps;
    L.tokens = tokens;
    L.K = K;
    L.codes = fmt->codes;
    L.gscale = fmt->group_scale;
    L.group = fmt->group;
    L.residual_out = residual_out;
    L.res_out_stride = res_out_stride;
    L.out_codes = codes;
    L.out_scales = gscales;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    return launched(launch_rmsnorm_quant(L), 1);
}

dq_status dq_kv_append(const void *k, int64_t k_token, int64_t k_head, const void *v, int64_t v_token,
                       int64_t v_head, int64_t tokens, const dq_kv_cache *cache,
                       const dq_kv_batch *batch, const dq_format *fmt, dq_stream stream) {
    return kv_copy(k, k_token, k_head, v, v_token, v_head, tokens, cache, batch, fmt, stream, false);
}

dq_status dq_kv_read(void *k, int64_t k_token, int64_t k_head, void *v, int64_t v_token, int64_t v_head,
                     int64_t tokens, const dq_kv_cache *cache, const dq_kv_batch *batch,
                     const dq_format *fmt, dq_stream stream) {
    return kv_copy(k, k_token, k_head, v, v_token, v_head, tokens, cache, batch, fmt, stream, true);
}

dq_status dq_kv_attention_workspace(int64_t tokens, int32_t q_heads, int32_t heads, int32_t head_dim,
                                    int32_t seqs, size_t *bytes) {
    if (!bytes) return DQ_ERR_ARG;
    if (tokens < 0 || tokens > INT32_MAX || seqs < 0 || heads <= 0 || heads > 65535 ||
        q_heads <= 0 || q_heads % heads || (head_dim != 64 && head_dim != 128))
        return DQ_ERR_SHAPE;
    *bytes = attend_workspace(tokens, q_heads, heads, head_dim, seqs);
    return DQ_OK;
}

dq_status dq_kv_attention(const void *q, int64_t q_token, int64_t q_head, void *out, int64_t out_token,
                          int64_t out_head, int64_t tokens, int32_t q_heads, float scale, int32_t causal,
                          const dq_kv_cache *cache, const dq_kv_batch *batch, const dq_format *fmt,
                          void *workspace, size_t ws_bytes, dq_stream stream) {
    dq_status s = check_cache(cache, batch, fmt, tokens);
    if (s != DQ_OK) return s;
    if (q_heads <= 0 || q_heads % cache->heads) return DQ_ERR_SHAPE;
    if (!(scale > 0.0f) || !std::isfinite(scale) || (causal != 0 && causal != 1)) return DQ_ERR_ARG;
    if (tokens == 0 || batch->seqs == 0) return DQ_OK;
    if (tokens * (q_heads / cache->heads) > INT32_MAX) return DQ_ERR_SHAPE;
    if ((s = check_rows(q, q_token, q_head, tokens, q_heads, cache->head_dim, false)) != DQ_OK) return s;
    if ((s = check_rows(out, out_token, out_head, tokens, q_heads, cache->head_dim, true)) != DQ_OK) return s;
    if (!workspace ||
        ws_bytes < attend_workspace(tokens, q_heads, cache->heads, cache->head_dim, batch->seqs))
        return DQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return DQ_ERR_ALIGN;
    // (rows of q are read until the call's end)
    if (overlap(q, q_token, q_head, out, out_token, out_head, tokens, q_heads, cache->head_dim)) return DQ_ERR_ARG;
    AttendLaunch L;
    L.status = serving_status_word();
    if (!L.status) return DQ_ERR_CUDA;
    L.q = q;
    L.q_token = q_token;
    L.q_head = q_head;
    L.out = out;
    L.out_token = out_token;
    L.out_head = out_head;
    L.tokens = tokens;
    L.q_heads = q_heads;
    L.scale = scale;
    L.causal = causal;
    L.cache = *cache;
    L.batch = *batch;
    L.codes = fmt->codes;
    L.gscale = fmt->group_scale;
    L.group = fmt->group;
    L.workspace = workspace;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    L.launches = 0;
    cudaError_t e;
    if (fmt->group_scale == DQ_SCALE_BF16) e = launch_attend_c0(L);
    else if (fmt->group_scale == DQ_SCALE_E4M3) e = launch_attend_c3(L);
    else if (fmt->codes == DQ_CODES_INT4) e = launch_attend_c1(L);
    else e = launch_attend_c2(L);
    return launched(e, L.launches);
}

}  // extern "C"
