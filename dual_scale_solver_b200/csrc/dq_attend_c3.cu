#include "dq_attend_prompt.cuh"

namespace dq {
cudaError_t launch_attend_c3(AttendLaunch &L) { return launch_attend_fmt<CODES_E2M1, SC_E4M3>(L); }
}  // namespace dq
