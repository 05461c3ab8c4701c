#include "dq_attend_prompt.cuh"

namespace dq {
cudaError_t launch_attend_c1(AttendLaunch &L) { return launch_attend_fmt<CODES_INT4, SC_E8M0>(L); }
}  // namespace dq
