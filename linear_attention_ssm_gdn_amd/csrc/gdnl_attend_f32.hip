// gdnl_attend_f32.hip -- the chunked kernels over fp32 rows.
#include "gdnl_attend.hpp"

namespace gdnl {

hipError_t launch_attend_f32(const AttendArgs& a, int mode, hipStream_t s) { return launch_attend<float>(a, mode, s); }

}  // namespace gdnl
