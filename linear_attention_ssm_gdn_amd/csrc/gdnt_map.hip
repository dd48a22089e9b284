// gdnt_map.hip -- the row map of a packed ragged batch, and the sum of
// per-tile partial gradients.
#include "gdnt_device.hpp"

namespace gdnt {

constexpr int kMapThreads = 256;

// The sequence that row r (< n_rows) is computed for, and its bounds; -1: none.
__device__ int owner(const MapArgs& A, int64_t r, bool bad, int& c0, int& c1) {
    int seq = -1;
    if (!bad) {
        int lo = 0, hi = A.n_seqs;  // the last s with cu[s] <= r, or -1
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)A.cu[mid] <= r) lo = mid + 1;
            else hi = mid;
        }
        seq = lo - 1;
        if (seq >= 0 && (int64_t)A.cu[seq + 1] <= r) seq = -1;
    } else {
        int end = 0;
        for (int s = 0; s < A.n_seqs; ++s) {
            const int b0 = A.cu[s], b1 = A.cu[s + 1];
            if (b0 < end || !bounds_ok(A.n_rows, b0, b1)) continue;
            if ((int64_t)b0 <= r && r < (int64_t)b1) { seq = s; break; }
            end = b1;
        }
    }
    if (seq < 0) return -1;
    c0 = A.cu[seq];
    c1 = A.cu[seq + 1];
    const int page = A.page_idx[seq];
    return page >= 0 && page < A.page_limit && (A.max_len == 0 || c1 - c0 <= A.max_len) ? seq : -1;
}

// One thread per row finds its sequence by bisection of cu_seqlens; every
// workgroup first looks all of cu_seqlens over (n_seqs / 256 loads a thread)
// and takes the slow scan where a bound is bad.  The first workgroup raises
// the error bits.  4 us for 2159 rows, 6.6 for 32768 with the 17 MB of chain
// words of 4096 channels to clear: about a launch.
__global__ __launch_bounds__(kMapThreads) void k_row_map(const MapArgs A) {
    const int tid = threadIdx.x;
    const int64_t gid = (int64_t)blockIdx.x * kMapThreads + tid;
    const int64_t stride = (int64_t)gridDim.x * kMapThreads;
    for (int64_t i = gid; i < A.n_zero; i += stride) A.zero[i] = 0;

    bool bad = false;
    for (int s = tid; s < A.n_seqs; s += kMapThreads) bad |= !bounds_ok(A.n_rows, A.cu[s], A.cu[s + 1]);
    bad = __syncthreads_or(bad) != 0;

    for (int64_t r = gid; r < A.n_map; r += stride) {
        int c0, c1;
        const int seq = r < A.n_rows ? owner(A, r, bad, c0, c1) : -1;
        A.map[r] = seq < 0 ? -1 : seq * 4 + (r == (int64_t)c1 - 1 ? 2 : 0) + (r == (int64_t)c0 ? 1 : 0);
    }

    if (blockIdx.x == 0) {
        for (int s = tid; s < A.n_seqs; s += kMapThreads) {
            const int page = A.page_idx[s];
            if (page < 0) continue;
            if (page >= A.page_limit) raise(A.err, GDN_DEVERR_PAGE);
            else if (bad && !valid_slow(A.cu, A.n_rows, s)) raise(A.err, GDN_DEVERR_BATCH);
            else if (A.max_len > 0 && A.cu[s + 1] - A.cu[s] > A.max_len) raise(A.err, GDN_DEVERR_BATCH);
        }
    }
    if (A.pass_dst) {  // rows of sequences that no kernel behind this one writes
        for (int s = blockIdx.x; s < A.n_seqs; s += gridDim.x) {
            const int page = A.page_idx[s], c0 = A.cu[s], c1 = A.cu[s + 1];
            const bool live = page >= 0 && page < A.page_limit && !(bad && !valid_slow(A.cu, A.n_rows, s)) &&
                              (A.max_len == 0 || c1 - c0 <= A.max_len);
            if (live && c0 != c1) continue;
            const int64_t at = (int64_t)s * A.pass_width;
            for (int64_t i = tid; i < A.pass_width; i += kMapThreads)
                A.pass_dst[at + i] = live && A.pass_src ? A.pass_src[at + i] : 0.0f;
        }
    }
}

hipError_t launch_map(const MapArgs& a, hipStream_t s) {
    // a workgroup clears up to 16 words a thread
    int64_t grid = (a.n_map + kMapThreads - 1) / kMapThreads;
    const int64_t by_zero = (a.n_zero + kMapThreads * 16 - 1) / (kMapThreads * 16);
    grid = grid > by_zero ? grid : by_zero;
    grid = grid < 1 ? 1 : grid > 4096 ? 4096 : grid;
    hipLaunchKernelGGL(k_row_map, dim3((unsigned)grid), dim3(kMapThreads), 0, s, a);
    return hipGetLastError();
}

// 64 channels by 16 groups of tiles to a workgroup; fp64, every order fixed.
// 4 to 6 us, a launch's time (19 MB of partial sums at 32768 x 8192).
constexpr int kSumGroups = 16;
__global__ __launch_bounds__(kSumGroups * 64) void k_sum_tiles(const float* part, int64_t n_tiles, int32_t C, int64_t Cp,
                                                               int n_out, float* out0, float* out1) {
    __shared__ double sum[kSumGroups][64];
    const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;  // < Cp
    const int j = blockIdx.y;
    double acc = 0.0;
#pragma unroll 4
    for (int64_t t = group; t < n_tiles; t += kSumGroups) acc += (double)part[(t * n_out + j) * Cp + c];
    sum[group][lane] = acc;
    __syncthreads();
    if (group == 0 && c < C) {
#pragma unroll
        for (int g = 1; g < kSumGroups; ++g) acc += sum[g][lane];
        const float v = (float)acc;
        if (out1) (j == 0 ? out0 : out1)[c] = v;
        else out0[c * n_out + j] = v;
    }
}

hipError_t launch_sum_tiles(const float* part, int64_t n_tiles, int32_t C, int n_out, float* out0, float* out1,
                            hipStream_t s) {
    const int64_t Cp = padded_channels(C);
    hipLaunchKernelGGL(k_sum_tiles, dim3((unsigned)(Cp / 64), (unsigned)n_out), dim3(kSumGroups * 64), 0, s, part, n_tiles, C, Cp,
                       n_out, out0, out1);
    return hipGetLastError();
}

}  // namespace gdnt
