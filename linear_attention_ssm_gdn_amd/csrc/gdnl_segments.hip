// gdnl_segments.hip -- which rows a workgroup of the chunked kernels walks,
// the states between segments, the gates' gradient and the sum over the value
// heads of a key head.
#include "gdn_device.hpp"
#include "gdnl_kernels.h"
#include "gdnt_device.hpp"

namespace gdnl {

using gdnt::bounds_ok;
using gdnt::raise;
using gdnt::valid_slow;

// The batch as the chunked kernels take it: which rows a slot's workgroups walk.
// Every workgroup first looks all of cu_seqlens over, and takes the slow check of
// a sequence's validity where a bound is bad.
struct Batch {
    const SegmentArgs& A;
    bool bad;
    __device__ __forceinline__ explicit Batch(const SegmentArgs& a) : A(a) {
        bool b = false;
        for (int s = threadIdx.x; s < A.n_seqs; s += kThreads) b |= !bounds_ok(A.n_rows, A.cu[s], A.cu[s + 1]);
        bad = __syncthreads_or(b) != 0;
    }
    __device__ __forceinline__ bool live(int s) const {
        const int page = A.page_idx[s];
        return page >= 0 && page < A.page_limit && !(bad && !valid_slow(A.cu, A.n_rows, s)) &&
               (A.max_len == 0 || A.cu[s + 1] - A.cu[s] <= A.max_len);
    }
    // One thread finds a slot's segment by bisection of cu_seqlens.
    __device__ __forceinline__ SegWord word_of(int64_t slot) const {
        // the last s with s + cu[s] / len <= slot; with a bad bound somewhere any valid s whose slots hold it
        int lo = 0, hi = A.n_seqs;
        if (!bad) {
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if ((int64_t)mid + A.cu[mid] / A.len <= slot) lo = mid + 1;
                else hi = mid;
            }
            hi = lo;
            lo = hi - 1;
        }
        for (int s = lo < 0 ? 0 : lo; s < hi; ++s) {
            const int c0 = A.cu[s], c1 = A.cu[s + 1];
            if (bad && !bounds_ok(A.n_rows, c0, c1)) continue;
            const int64_t at = slot - ((int64_t)s + c0 / A.len);
            if (at < 0 || at * A.len >= c1 - c0 || !live(s)) continue;
            const int row = c0 + (int)at * A.len, rows = c1 - row < A.len ? c1 - row : A.len;
            return SegWord{s, row, rows, A.page_idx[s] * 4 + (row + rows == c1 ? 2 : 0) + (at == 0 ? 1 : 0)};
        }
        return SegWord{0, 0, 0, 0};
    }
    // All that is not of a slot, by the whole grid.
    __device__ __forceinline__ void rest() const {
        const int tid = threadIdx.x;
        const int64_t gid = (int64_t)blockIdx.x * kThreads + tid, stride = (int64_t)gridDim.x * kThreads;
        for (int64_t s = gid; s < A.n_seqs; s += stride) {
            const bool ok = live((int)s);
            const int len = ok ? A.cu[s + 1] - A.cu[s] : 0;
            A.seqs[s] = SeqSlots{ok ? (int)s + A.cu[s] / A.len : 0, ok ? (int)(((int64_t)len + A.len - 1) / A.len) : 0};
        }
        if (blockIdx.x == 0) {
            for (int s = tid; s < A.n_seqs; s += kThreads) {
                const int page = A.page_idx[s];
                if (page < 0) continue;
                if (page >= A.page_limit) raise(A.err, GDN_DEVERR_PAGE);
                else if (bad && !valid_slow(A.cu, A.n_rows, s)) raise(A.err, GDN_DEVERR_BATCH);
                else if (A.max_len > 0 && A.cu[s + 1] - A.cu[s] > A.max_len) raise(A.err, GDN_DEVERR_BATCH);
            }
        }
        if (A.pass_dst) {  // gradients of sequences that no kernel behind this one writes
            const int64_t parts = gridDim.x > A.n_seqs ? gridDim.x / A.n_seqs : 1;  // workgroups to a sequence
            for (int64_t u = blockIdx.x; u < A.n_seqs * parts; u += gridDim.x) {
                const int s = (int)(u / parts);
                const bool ok = live(s);
                if (ok && A.cu[s] != A.cu[s + 1]) continue;
                const int64_t at = (int64_t)s * A.pass_width;
                for (int64_t j = u % parts * kThreads + tid; j < A.pass_width; j += parts * kThreads)
                    A.pass_dst[at + j] = ok && A.pass_src ? A.pass_src[at + j] : 0.0f;
            }
        }
    }
};

// A thread to a slot.  About a launch's time, 5 us.
__global__ __launch_bounds__(kThreads) void k_segments(const SegmentArgs A) {
    const Batch batch(A);
    for (int64_t slot = (int64_t)blockIdx.x * kThreads + threadIdx.x; slot < A.n_slots; slot += (int64_t)gridDim.x * kThreads)
        A.segs[slot] = batch.word_of(slot);
    batch.rest();
}

hipError_t launch_segments(const SegmentArgs& a, hipStream_t s) {
    int64_t n = a.n_slots > a.n_seqs ? a.n_slots : a.n_seqs;
    int64_t grid = (n + kThreads - 1) / kThreads;
    if (a.pass_dst && grid < a.n_seqs) grid = a.n_seqs;
    grid = grid < 1 ? 1 : grid > 1024 ? 1024 : grid;
    hipLaunchKernelGGL(k_segments, dim3((unsigned)grid), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

// 2^x for x = n + f, |f| <= 1/2: 2^f = 1 + f (c_0 + c_1 f + ...), where
// c_k = log(2)^{k+1} / (k+1)! and the rest after nine terms is below 2^-35; the
// last product and sum in F's precision (in fp32 within 0.6 of its last bit).
template <class F> __device__ __forceinline__ F exp2_of(double x) {
    const double n = rint(x);
    const F f = fabs(x) > 2000.0 ? F(0) : F(x - n);  // 0 or infinite, whatever f is
    F p = F(1.0178086e-7);
    p = fma(p, f, F(1.3215486790e-6));
    p = fma(p, f, F(1.52527338041e-5));
    p = fma(p, f, F(1.54035303934e-4));
    p = fma(p, f, F(1.33335581464e-3));
    p = fma(p, f, F(9.61812910763e-3));
    p = fma(p, f, F(5.55041086648e-2));
    p = fma(p, f, F(0.240226506959101));
    p = fma(p, f, F(0.693147180559945));
    return ldexp(fma(f, p, F(1)), (int)fmin(fmax(n, -1000.0), 1000.0));
}

// A workgroup to a segment and head, a wave to a chunk, a lane to a row.  g ends
// at -128, where e^g is 0: differences of the sums behind it stay finite.
//
// e^{G_C}, by which the state is multiplied at every chunk, takes up what rounding
// it left of the chunks before: their product is then off by one rounding however
// many they are, and not by one for each, all to the same side where decays are
// fixed.  16-22 us over 32768 rows of 32 heads.
__device__ __forceinline__ void decays_of(const DecayArgs& A, const int4& w, int head) {
    constexpr int kWaves = kThreads / 64;
    __shared__ double s_sum[kWaves], s_whole[2][kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (w.z <= 0) return;
    double total = 0.0;
    float left = 0.0f;  // of the product of the chunks' factors, relative
    for (int t0 = 0, turn = 0; t0 < w.z; t0 += kThreads, turn ^= 1) {
        const int t = t0 + threadIdx.x;
        const int64_t row = (int64_t)w.y + t;
        const bool in = t < w.z;
        const float g = in ? A.g[row * A.g_stride + head] : 0.0f;
        double G = (double)(g < -128.0f ? -128.0f : g) * 1.4426950408889634;  // a NaN stays
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double up = __shfl_up(G, d, 64);
            if (lane >= d) G += up;
        }
        const double GC = __shfl(G, 63, 64);
        total += GC;
        if (lane == 0) s_whole[turn][wave] = exp2_of<double>(GC);
        __syncthreads();
        float whole = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            const double exact = s_whole[turn][k] * (1.0 + (double)left);
            const float f = (float)exact;
            left = f > 1.0e-30f && f < __builtin_inff() ? (float)(exact - (double)f) / f : 0.0f;
            if (k == wave) whole = f;
        }
        const float hi = (float)G, lo = (float)(G - (double)hi);
        const bool last = lane == 63 || t == w.z - 1;
        if (in)
            A.gates[(int64_t)head * A.n_rows + row] =
                make_float4(hi, lo, last ? whole : exp2_of<float>(G), exp2_of<float>(GC - G));
    }
    if (lane == 0) s_sum[wave] = total;
    __syncthreads();
    if (threadIdx.x == 0) A.total[blockIdx.x] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}
__global__ __launch_bounds__(kThreads) void k_decays(const DecayArgs A) {
    decays_of(A, *reinterpret_cast<const int4*>(A.segs + blockIdx.x / A.heads), (int)(blockIdx.x % A.heads));
}

// Both in one launch where sequences are few enough for every workgroup to find
// its own segment: 8.3 us against 4.7 and 6.0 for 8 sequences of 2159 rows and 32
// heads, a call over 63 rows 17.2 us against 19.9.
constexpr int kFewSeqs = 256;
__global__ __launch_bounds__(kThreads) void k_segments_decays(const SegmentArgs S, const DecayArgs A) {
    __shared__ alignas(16) SegWord s_word;
    const Batch batch(S);
    const int64_t slot = blockIdx.x / A.heads;
    const int head = (int)(blockIdx.x % A.heads);
    if (threadIdx.x == 0) {
        s_word = batch.word_of(slot);
        if (head == 0) S.segs[slot] = s_word;
    }
    batch.rest();
    __syncthreads();
    decays_of(A, *reinterpret_cast<const int4*>(&s_word), head);
}
hipError_t launch_segments_decays(const SegmentArgs& s, const DecayArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.n_slots * a.heads));
    if (s.n_seqs <= kFewSeqs) {
        hipLaunchKernelGGL(k_segments_decays, grid, dim3(kThreads), 0, stream, s, a);
        return hipGetLastError();
    }
    const hipError_t e = launch_segments(s, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_decays, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

// The states at borders.  A lane holds a value of the state, and a wave eight
// borders of the round, whose local sums it asks for together; with more borders
// than that, waves of a workgroup take eight each, fold them to (decay, sum), and
// each takes its state from the folds before it.  One round of loads and one of
// stores for 128 borders: 36 us -> 8 us for 118 segments of four heads of 64 x 64,
// where waiting is all of it; 28 us for 16 segments of 4 x 32 heads of 128 x 128.
constexpr int kScanMine = 8, kScanWaves = 16;
__global__ __launch_bounds__(kScanWaves * 64) void k_state_scan(const ScanArgs A, int blocks, int waves, int width) {
    __shared__ float s_sum[kScanWaves][64], s_decay[kScanWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int mine = wave % waves, team = wave / waves * waves;  // of the waves that share 64 values
    for (int64_t b = blockIdx.x; b < (int64_t)A.n_seqs * A.heads * blocks; b += gridDim.x) {
        const int part = (int)(b % blocks), head = (int)(b / blocks % A.heads), seq = (int)(b / blocks / A.heads);
        const SeqSlots at = A.seqs[seq];
        const int e = part * width + team / waves * 64 + lane;
        const int n = at.n - 1;  // borders
        if (n <= 0) continue;
        const bool in = e < A.size;
        const bool zero = A.in.at == kNoState || (A.in.at == kByPage && A.has_init && A.has_init[seq] == 0);
        float carry = 0.0f;
        if (in && !zero) {
            const int64_t from = (A.in.at == kByPage ? (int64_t)A.page_idx[seq] : (int64_t)seq) * A.in.unit + head * A.in.head + e;
            carry = A.in.bf16 ? gdn::to_f32(static_cast<const gdn::bf16_t*>(A.in.p)[from]) : static_cast<const float*>(A.in.p)[from];
        }
        if (A.copy && in && mine == 0) A.copy[((int64_t)(at.slot - seq) * A.heads + head) * A.size + e] = carry;
        const int64_t step = A.back ? -A.heads : A.heads;
        for (int k0 = 0; k0 < n; k0 += kScanMine * waves) {
            const int first = k0 + mine * kScanMine;
            // the segment whose local sum is at the border, and the border: slot - seq is that of the first row
            const int64_t item = (int64_t)(at.slot + (A.back ? n : 0)) * A.heads + head + step * first;
            const int64_t border = (int64_t)(at.slot - seq + (A.back ? n : 1)) * A.heads + head + step * first;
            float own[kScanMine], factor[kScanMine];
#pragma unroll
            for (int j = 0; j < kScanMine; ++j)
                own[j] = first + j < n && in ? A.local[(border + step * j) * A.size + e] : 0.0f;
            // the factors, each made by a lane, take up what rounding left of those before, as in decays_of
            const int j8 = lane % kScanMine;
            const double exact = exp2_of<double>(first + j8 < n ? A.total[item + step * j8] : 0.0);
            const float exact_hi = (float)exact, exact_lo = fabsf(exact_hi) < __builtin_inff() ? (float)(exact - (double)exact_hi) : 0.0f;
            float left = 0.0f;
#pragma unroll
            for (int j = 0; j < kScanMine; ++j) {
                const float hi = __shfl(exact_hi, j, 64), rest = fmaf(hi, left, __shfl(exact_lo, j, 64));
                factor[j] = hi + rest;
                left = factor[j] > 1.0e-30f && factor[j] < __builtin_inff() ? ((hi - factor[j]) + rest) * gdnt::rcp(factor[j]) : 0.0f;
            }
            float cur = carry;
            if (waves > 1) {
                float sum = 0.0f, decay = 1.0f;
#pragma unroll
                for (int j = 0; j < kScanMine; ++j) {
                    sum = fmaf(factor[j], sum, own[j]);
                    decay *= factor[j];
                }
                __syncthreads();  // the round before has been read
                s_sum[wave][lane] = sum;
                if (lane == 0) s_decay[wave] = decay;
                __syncthreads();
                for (int w = 0; w < waves; ++w) {
                    if (w == mine) cur = carry;
                    carry = fmaf(s_decay[team + w], carry, s_sum[team + w][lane]);
                }
            }
#pragma unroll
            for (int j = 0; j < kScanMine; ++j) {
                cur = fmaf(factor[j], cur, own[j]);
                if (in && first + j < n) A.local[(border + step * j) * A.size + e] = cur;
            }
            if (waves == 1) carry = cur;
        }
    }
}
hipError_t launch_state_scan(const ScanArgs& a, int64_t segments, hipStream_t s) {
    int waves = 1;  // a power of two, so that teams fill the workgroup
    while (waves < kScanWaves && (int64_t)waves * kScanMine < segments) waves *= 2;
    const int threads = waves > 4 ? waves * 64 : kThreads, width = threads / waves;
    const int blocks = (a.size + width - 1) / width;
    int64_t grid = (int64_t)a.n_seqs * a.heads * blocks;
    if (grid > (1 << 20)) grid = 1 << 20;
    hipLaunchKernelGGL(k_state_scan, dim3((unsigned)grid), dim3((unsigned)threads), 0, s, a, blocks, waves, width);
    return hipGetLastError();
}

template <int W> __device__ __forceinline__ double block_sum(double v, double* s_part) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = v;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) all += s_part[w];
    return all;
}

// <state, its gradient> behind every segment, and in front of every sequence:
// a workgroup to a pair of states.  Bound by their bytes: 15 us for 512 pairs of
// 128 x 128 (67 MB at 4.5 TB/s).
constexpr int kEndThreads = 1024;
__global__ __launch_bounds__(kEndThreads) void k_gate_ends(const GateArgs A) {
    __shared__ double s_part[kEndThreads / 64];
    const int tid = threadIdx.x;
    for (int64_t b = blockIdx.x; b < (A.n_slots + A.n_seqs) * A.heads; b += gridDim.x) {
        const int64_t unit = b / A.heads;
        const int head = (int)(b % A.heads);
        const float* e = nullptr;
        States p{};
        int64_t at = 0;
        if (unit < A.n_slots) {
            const int4 w = *reinterpret_cast<const int4*>(A.segs + unit);
            if (w.z > 0 && (w.w & 2) != 0 && A.d_state) {
                p.p = const_cast<float*>(A.last);
                at = ((int64_t)w.x * A.heads + head) * A.size;
                e = A.d_state + at;
            } else if (w.z > 0 && (w.w & 2) == 0) {
                p.p = const_cast<float*>(A.before);
                at = ((int64_t)(w.y / A.len + 1) * A.heads + head) * A.size;
                e = A.after + at;
            }
        } else {
            const int seq = (int)(unit - A.n_slots);
            if (A.seqs[seq].n > 0 && !(A.has_init && A.has_init[seq] == 0)) {
                p = A.start;
                at = (int64_t)A.page_idx[seq] * p.unit + head * p.head;
                e = A.first + ((int64_t)seq * A.heads + head) * A.size;
            }
        }
        double x = 0.0;
        if (e && p.bf16) {
            for (int j = tid; j < A.size; j += kEndThreads)
                x += (double)gdn::to_f32(static_cast<const gdn::bf16_t*>(p.p)[at + j]) * (double)e[j];
        } else if (e) {
#pragma unroll 8
            for (int j = tid; j < A.size; j += kEndThreads) x += (double)static_cast<const float*>(p.p)[at + j] * (double)e[j];
        }
        x = block_sum<kEndThreads / 64>(x, s_part);
        if (tid == 0) A.ends[b] = x;
    }
}

// A workgroup to a segment and head: the gradients of its decays, 256 rows at a
// time from the last, in 64 bits.  That of row t is X behind the segment and what
// the rows from t on bring, rows - cols.  Summed over the segment they have to
// end at X in front of it; what they miss it by, the rounding of hundreds of
// products, is spread over the rows in the measure of what they bring.  Errors
// then stay those of a walk that is held at both ends, and a decay's own
// rounding, the same in every chunk where decays are fixed, cancels: 1.3e-6 -> 7e-7
// of the gradients' norm over 4 x 8192 rows; summed over 2472 rows of six fixed
// decays, twelve draws, 1.3e-6 -> 3.2e-7.
__global__ __launch_bounds__(kThreads) void k_gate(const GateArgs A) {
    __shared__ double s_part[4];
    __shared__ double s_wave[4];
    const int64_t slot = blockIdx.x / A.heads;
    const int head = (int)(blockIdx.x % A.heads), tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int4 w = *reinterpret_cast<const int4*>(A.segs + slot);
    const int row0 = w.y, rows = w.z;
    if (rows <= 0) {
        if (A.part && tid == 0) A.part[blockIdx.x] = 0.0;
        return;
    }
    const float* const in = A.rows + (int64_t)head * A.n_rows + row0;
    const float* const out = A.cols + (int64_t)head * A.n_rows + row0;
    double carry = A.ends[blockIdx.x], sum = 0.0;
    const double front_x = A.ends[((w.w & 1) != 0 ? A.n_slots + w.x : slot - 1) * A.heads + head];
    double all = 0.0, size = 0.0;
    for (int t = tid; t < rows; t += kThreads) {
        all += (double)in[t] - (double)out[t];
        size += (double)(fabsf(in[t]) + fabsf(out[t]));
    }
    all = block_sum<4>(all, s_part);
    size = block_sum<4>(size, s_part);
    const double missed = size > 0.0 ? (front_x - carry - all) / size : 0.0;
    for (int t0 = (rows - 1) / kThreads * kThreads; t0 >= 0; t0 -= kThreads) {
        // thread 0 takes the tile's last row
        const int t = t0 + kThreads - 1 - tid;
        double v = 0.0;
        if (t < rows) v = ((double)in[t] - (double)out[t]) + missed * (double)(fabsf(in[t]) + fabsf(out[t]));
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double up = __shfl_up(v, d, 64);
            if (lane >= d) v += up;
        }
        __syncthreads();
        if (lane == 63) s_wave[wave] = v;
        __syncthreads();
        double front = carry;
        for (int k = 0; k < 4; ++k) {
            if (k < wave) front += s_wave[k];
            carry += s_wave[k];
        }
        if (t < rows) {
            // a decay of 0 lets no gradient through
            const float gv = A.g[((int64_t)row0 + t) * A.g_stride + head];
            const double dg = gv < -128.0f ? 0.0 : front + v;
            if (A.part) sum += dg;
            else A.dg[((int64_t)row0 + t) * A.heads + head] = (float)dg;
        }
    }
    if (A.part) {
        sum = block_sum<4>(sum, s_part);
        if (tid == 0) A.part[blockIdx.x] = sum;
    }
}
hipError_t launch_gate(const GateArgs& a, hipStream_t s) {
    const int64_t pairs = (a.n_slots + a.n_seqs) * a.heads;
    hipLaunchKernelGGL(k_gate_ends, dim3((unsigned)(pairs < (1 << 16) ? pairs : 1 << 16)), dim3(kEndThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_gate, dim3((unsigned)(a.n_slots * a.heads)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

__global__ __launch_bounds__(kThreads) void k_gate_sum(const double* part, int64_t n_slots, int32_t heads, float* dg) {
    __shared__ double s_part[4];
    double v = 0.0;
    for (int64_t j = threadIdx.x; j < n_slots; j += kThreads) v += part[j * heads + blockIdx.x];
    v = block_sum<4>(v, s_part);
    if (threadIdx.x == 0) dg[blockIdx.x] = (float)v;
}
hipError_t launch_gate_sum(const double* part, int64_t n_slots, int32_t heads, float* dg, hipStream_t s) {
    hipLaunchKernelGGL(k_gate_sum, dim3((unsigned)heads), dim3(kThreads), 0, s, part, n_slots, heads, dg);
    return hipGetLastError();
}

// Four rows of a segment to a workgroup at a time, V values to a thread.  Bound by
// bytes: 132 us over 32768 rows of 32 heads of 128 (5.1 TB/s).
constexpr int kGroupRows = 4;
template <int V> __global__ __launch_bounds__(kThreads) void k_group_sum(const GroupArgs A, int blocks) {
    const int64_t slot = blockIdx.x / blocks;
    const int4 w = *reinterpret_cast<const int4*>(A.segs + slot);
    const int per_row = A.heads / A.per * (A.d / V), per_head = A.d / V;
    for (int t0 = (int)(blockIdx.x % blocks) * kGroupRows; t0 < w.z; t0 += blocks * kGroupRows) {
        const int n = min(kGroupRows, w.z - t0);
        for (int j = threadIdx.x; j < n * per_row; j += kThreads) {
            const int t = j / per_row, c = j - t * per_row, h = c / per_head, d = (c - h * per_head) * V;
            const int64_t row = (int64_t)w.y + t0 + t;
            const float* p = A.part + (row * A.heads + (int64_t)h * A.per) * A.d + d;
            float v[V] = {};
            for (int q = 0; q < A.per; ++q) {
                if constexpr (V == 4) {
                    const float4 u = *reinterpret_cast<const float4*>(p + (int64_t)q * A.d);
                    v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
                } else {
                    v[0] += p[(int64_t)q * A.d];
                }
            }
            const int64_t at = row * A.stride + (int64_t)h * A.d + d;
            if constexpr (V == 4) {
                if (A.bf16) gdnt::store4<true>(static_cast<gdn::bf16_t*>(A.out) + at, v, 4);
                else gdnt::store4<true>(static_cast<float*>(A.out) + at, v, 4);
            } else {
                if (A.bf16) static_cast<gdn::bf16_t*>(A.out)[at] = gdn::f32_to_bf16(v[0]);
                else static_cast<float*>(A.out)[at] = v[0];
            }
        }
    }
}
hipError_t launch_group_sum(const GroupArgs& a, hipStream_t s) {
    // as many workgroups as a segment has rows for, within some 16384
    int64_t blocks = (a.most_rows + kGroupRows - 1) / kGroupRows;
    const int64_t most = 16384 / a.n_slots + 1;
    blocks = blocks > most ? most : blocks < 1 ? 1 : blocks;
    const dim3 grid((unsigned)(a.n_slots * blocks)), block(kThreads);
    if (a.vec) hipLaunchKernelGGL(k_group_sum<4>, grid, block, 0, s, a, (int)blocks);
    else hipLaunchKernelGGL(k_group_sum<1>, grid, block, 0, s, a, (int)blocks);
    return hipGetLastError();
}

}  // namespace gdnl
