// gdnl_attend_f32_back.hip -- the chunked kernels over fp32 rows: backward in time.
#include "gdnl_attend.hpp"

namespace gdnl {

hipError_t launch_attend_f32_back(const AttendArgs& a, int mode, hipStream_t s) {
    if (mode == kAttend) return launch_attend<float, kAttend, true>(a, s);
    return mode == kDot ? launch_attend<float, kDot, true>(a, s) : launch_attend<float, kLocal, true>(a, s);
}

}  // namespace gdnl
