#include "dq_attend_prompt.cuh"

namespace dq {

size_t attend_workspace(int64_t tokens, int32_t q_heads, int32_t heads, int32_t head_dim, int32_t seqs) {
    (void)tokens, (void)q_heads, (void)heads, (void)seqs;
    return (size_t)2 * kAttCtas * kAttRowsMax * (head_dim * sizeof(float) + sizeof(float2)) +
           kAttCtas * sizeof(AttMeta);
}

cudaError_t launch_attend_c0(AttendLaunch &L) { return launch_attend_fmt<CODES_INT4, SC_BF16>(L); }
}  // namespace dq
