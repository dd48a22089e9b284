// gdnl_attend_bf16.hip -- the chunked kernels over bf16 rows: forward in time.
#include "gdnl_attend.hpp"

namespace gdnl {

hipError_t launch_attend_bf16(const AttendArgs& a, int mode, hipStream_t s) {
    if (mode == kAttend) return launch_attend<bf16_t, kAttend, false>(a, s);
    return mode == kDotRows ? launch_attend<bf16_t, kDotRows, false>(a, s) : launch_attend<bf16_t, kLocal, false>(a, s);
}

}  // namespace gdnl
