// gdnl_attend_f32.hip -- the chunked kernels over fp32 rows: forward in time.
#include "gdnl_attend.hpp"

namespace gdnl {

hipError_t launch_attend_f32(const AttendArgs& a, int mode, hipStream_t s) {
    if (mode == kAttend) return launch_attend<float, kAttend, false>(a, s);
    return mode == kDotRows ? launch_attend<float, kDotRows, false>(a, s) : launch_attend<float, kLocal, false>(a, s);
}

}  // namespace gdnl
