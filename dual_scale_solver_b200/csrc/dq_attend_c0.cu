#include "dq_attend_prompt.cuh"

namespace dq {

size_t attend_workspace(int64_t tokens, int32_t q_heads, int32_t heads, int32_t head_dim, int32_t seqs) {
    // two pieces per CTA: rows of float32 sums with their (maximum, sum)
    const size_t row = head_dim * sizeof(float) + sizeof(float2);
    // (calls of both kernels use it one after the other)
    return attend_kernels(tokens, q_heads, heads, seqs) & ATT_MANY
               ? 2 * kPromptCtas * kPromptRows * row + kPromptCtas * sizeof(AttMeta)
               : 2 * kAttCtas * 8 * row + kAttCtas * sizeof(AttMeta);
}

cudaError_t launch_attend_c0(AttendLaunch &L) { return launch_attend_fmt<CODES_INT4, SC_BF16>(L); }
}  // namespace dq
