// gdnl_tokens.hip -- linear attention row by row: sequences of a few rows, one
// workgroup to a sequence and value head.
//
// The state passes through the registers once: a wave takes two rows of up to
// 128 columns at a time, four columns a lane, so a load is a run of 1 KB, and
// all of a head's 64 KB are asked for before the first is used.  A row costs
//   S <- e^g S + k v^T,  o = scale S^T q,
// each lane its 16 rows, then a sum over the eight row groups through LDS.
// Bound by the state's bytes, read and written once: 64 sequences of 32 heads of
// 128 x 128 in fp32 take 47 us, 268 MB at 5.7 TB/s.
#include "gdn_device.hpp"
#include "gdnl_kernels.h"
#include "gdnt_device.hpp"

namespace gdnl {

using gdn::bf16_t;
using gdnt::bounds_ok;
using gdnt::raise;
using gdnt::valid_slow;

// COLS: 64 or 128 columns side by side.
template <typename T, typename S, int COLS, bool VEC>
__global__ __launch_bounds__(kThreads) void k_tokens(const TokenArgs A) {
    constexpr int kLanes = COLS / 4, kGroups = kThreads / kLanes, kMine = kMaxDim / kGroups;
    __shared__ float s_q[kMaxDim], s_k[kMaxDim], s_o[kGroups][COLS];
    const int tid = threadIdx.x;
    const int seq = (int)(blockIdx.x / A.heads), head = (int)(blockIdx.x % A.heads);
    const int page = A.page_idx[seq];
    if (page < 0) return;
    const int c0 = A.cu[seq], c1 = A.cu[seq + 1];
    bool bad = false;
    for (int s = tid; s <= seq; s += kThreads) bad |= !bounds_ok(A.n_rows, A.cu[s], A.cu[s + 1]);
    bad = __syncthreads_or(bad) != 0;
    uint32_t refused = 0;
    if (page >= A.page_limit) refused = GDN_DEVERR_PAGE;
    else if (bad && !valid_slow(A.cu, A.n_rows, seq)) refused = GDN_DEVERR_BATCH;
    else if (c1 - c0 > A.max_len) refused = GDN_DEVERR_BATCH;
    if (refused) {
        if (head == 0 && tid == 0) raise(A.err, refused);
        return;
    }
    if (c0 == c1) return;

    const int col = tid % kLanes * 4, grp = tid / kLanes;
    const int nc = A.dv - col;  // columns of this lane that exist: nc >= 4, or fewer
    const bool init = !A.has_init || A.has_init[seq] != 0;
    const S* in = static_cast<const S*>(A.st_in) + (int64_t)page * A.st_in_stride + (int64_t)head * A.dk * A.dv;
    S* out = static_cast<S*>(A.st_out) + (int64_t)page * A.st_out_stride + (int64_t)head * A.dk * A.dv;
    float st[kMine][4];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int row = m * kGroups + grp;
        gdnt::Raw4<S> raw = gdnt::zero4<S>();
        if (init && row < A.dk && nc > 0) raw = gdnt::load4<S, VEC>(in + (int64_t)row * A.dv + col, nc < 4 ? nc : 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) st[m][j] = raw.get(j);
    }
    for (int t = c0; t < c1; ++t) {
        const T* q = static_cast<const T*>(A.q) + t * A.q_stride + (int64_t)(head / A.per) * A.dk;
        const T* k = static_cast<const T*>(A.k) + t * A.k_stride + (int64_t)(head / A.per) * A.dk;
        const T* v = static_cast<const T*>(A.v) + t * A.v_stride + (int64_t)head * A.dv + col;
        const float g = A.g[t * A.g_stride + head];
        if (tid < A.dk) s_k[tid] = gdn::to_f32(k[tid]);
        else if (tid >= kMaxDim && tid - kMaxDim < A.dk) s_q[tid - kMaxDim] = gdn::to_f32(q[tid - kMaxDim]);
        float vv[4], o[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) vv[j] = j < nc ? gdn::to_f32(v[j]) : 0.0f;
        const float decay = g < -128.0f ? 0.0f : expf(g);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int row = m * kGroups + grp;
            if (row < A.dk) {
                const float kr = s_k[row], qr = s_q[row];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    st[m][j] = fmaf(kr, vv[j], decay * st[m][j]);
                    o[j] = fmaf(qr, st[m][j], o[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s_o[grp][col + j] = o[j];
        __syncthreads();
        if (tid < COLS && tid < A.dv) {
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < kGroups; ++r) sum += s_o[r][tid];
            static_cast<T*>(A.o)[t * A.o_stride + (int64_t)head * A.dv + tid] = gdn::from_f32<T>(A.scale * sum);
        }
    }
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int row = m * kGroups + grp;
        if (row < A.dk && nc > 0) gdnt::store4<VEC>(out + (int64_t)row * A.dv + col, st[m], nc < 4 ? nc : 4);
    }
}

template <typename T, typename S> hipError_t run_tokens(const TokenArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.n_seqs * a.heads)), block(kThreads);
    if (a.dv <= 64) {
        if (a.vec) hipLaunchKernelGGL((k_tokens<T, S, 64, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_tokens<T, S, 64, false>), grid, block, 0, s, a);
    } else {
        if (a.vec) hipLaunchKernelGGL((k_tokens<T, S, 128, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_tokens<T, S, 128, false>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}
hipError_t launch_tokens(const TokenArgs& a, hipStream_t s) {
    if (a.act_bf16) return a.state_bf16 ? run_tokens<bf16_t, bf16_t>(a, s) : run_tokens<bf16_t, float>(a, s);
    return a.state_bf16 ? run_tokens<float, bf16_t>(a, s) : run_tokens<float, float>(a, s);
}

}  // namespace gdnl
