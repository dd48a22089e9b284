// gdnl_attend_bf16.hip -- the chunked kernels over bf16 rows.
#include "gdnl_attend.hpp"

namespace gdnl {

hipError_t launch_attend_bf16(const AttendArgs& a, int mode, hipStream_t s) { return launch_attend<bf16_t>(a, mode, s); }

}  // namespace gdnl
