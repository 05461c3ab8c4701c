#include "dq_attend_prompt.cuh"

namespace dq {
cudaError_t launch_attend_c2(AttendLaunch &L) { return launch_attend_fmt<CODES_E2M1, SC_E8M0>(L); }
}  // namespace dq
