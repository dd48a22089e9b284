// gdnl_attend_bf16_back.hip -- the chunked kernels over bf16 rows: backward in time.
#include "gdnl_attend.hpp"

namespace gdnl {

hipError_t launch_attend_bf16_back(const AttendArgs& a, int mode, hipStream_t s) {
    if (mode == kAttend) return launch_attend<bf16_t, kAttend, true>(a, s);
    return mode == kDot ? launch_attend<bf16_t, kDot, true>(a, s) : launch_attend<bf16_t, kLocal, true>(a, s);
}

}  // namespace gdnl
