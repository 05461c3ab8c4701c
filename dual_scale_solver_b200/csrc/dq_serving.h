// dq_serving.h — host-side launch entry points of the serving operators (the
// C ABI of include/dq_serving.h) and what they share with dq_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dq_serving.h"

namespace dq {

constexpr unsigned int STATUS_INDEX = 8u;      // device flag read as DQ_ERR_INDEX

// dq_api.cu: the current device's flag word, the launch counter, format checks
unsigned int *serving_status_word();
void serving_count_launches(int k);
dq_status serving_format(const dq_format *f, int *bits);

// ---- residual + root-mean-square norm + quantization (dq_rmsnorm.cu)
struct NormLaunch {
    const void *x, *residual;       // bf16 rows (residual may be NULL)
    int64_t x_stride, res_stride;   // elements between rows
    const void *weight;             // [K], float32 or bf16
    int weight_f32;
    const float *b;                 // [K] or NULL
    float eps;
    int64_t tokens, K;
    int codes, gscale, group;       // DQ_CODES_*, DQ_SCALE_*, G
    void *residual_out;             // bf16 rows or NULL
    int64_t res_out_stride;
    uint8_t *out_codes;
    void *out_scales;
    unsigned int *status;
    cudaStream_t stream;
};
cudaError_t launch_rmsnorm_quant(const NormLaunch &L);

// ---- the 4-bit cache (dq_kv_cache.cu)
struct KvCopyLaunch {
    const void *k, *v;              // bf16 token arrays (read: written)
    int64_t k_token, k_head, v_token, v_head;
    int64_t tokens;
    dq_kv_cache cache;
    dq_kv_batch batch;
    int codes, gscale, group;
    unsigned int *status;
    cudaStream_t stream;
};
cudaError_t launch_kv_append(const KvCopyLaunch &L);
cudaError_t launch_kv_read(const KvCopyLaunch &L);

// ---- attention over the cache
struct AttendLaunch {
    const void *q;
    int64_t q_token, q_head;
    void *out;
    int64_t out_token, out_head;
    int64_t tokens;
    int32_t q_heads;
    float scale;
    int32_t causal;
    dq_kv_cache cache;
    dq_kv_batch batch;
    int codes, gscale, group;
    void *workspace;
    unsigned int *status;
    cudaStream_t stream;
    int launches;                   // out: kernels launched
};
// workspace of a launch (any of the kernels)
size_t attend_workspace(int64_t tokens, int32_t q_heads, int32_t heads, int32_t head_dim,
                        int32_t seqs);
cudaError_t launch_attend_c0(AttendLaunch &L);   // INT4, BF16 group scales
cudaError_t launch_attend_c1(AttendLaunch &L);   // INT4, E8M0
cudaError_t launch_attend_c2(AttendLaunch &L);   // E2M1, E8M0
cudaError_t launch_attend_c3(AttendLaunch &L);   // E2M1, E4M3

}  // namespace dq
