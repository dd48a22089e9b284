// gdnl_rotate.hip -- the norm of every head of q and k and its rotation by
// position in one pass, and its backward pass.
//
// A head's d values are d/2 pairs: (i, i + rot/2) or (2i, 2i + 1) among the
// first `rot`, neighbours behind them, which are not turned.  Sixteen lanes
// hold a head, VEC pairs of them side by side, so that both halves of a pair
// are in one lane and a norm is one sum over a DPP row.
//
// The angle pos * inv_freq is an fp64 product, reduced to a fraction of a turn
// in fp64 (for a position of 10^6 its last digits in fp32 are half a radian),
// and its sine and cosine are made once for a row, for all its heads, in LDS:
// those of the fraction in fp32, and to first order what that rounding left.
//
// Bound by the bytes of x and y: 32768 rows of 48 heads of 128 in bf16 take 146-172
// us forward (5.1 TB/s at the middle) and 280-349 us backward.
#include "gdn_device.hpp"
#include "gdnl_kernels.h"

namespace gdnl {

using gdn::bf16_t;
using gdn::reduce16;

constexpr int kLanes = 16, kHeadsAtOnce = kThreads / kLanes;
constexpr int kMaxPairs = 128;  // of a head
constexpr int kRotRows = 4;     // rows whose angles stand in LDS together

// Pairs p0..p0+N-1 of a head at x: first and second values.
template <typename T, int N> struct Pairs {
    float a[N], b[N];
};
__device__ __forceinline__ void unpack(uint2 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void get4(const bf16_t* p, float (&f)[4]) { unpack(*reinterpret_cast<const uint2*>(p), f); }
__device__ __forceinline__ void get4(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
__device__ __forceinline__ void put4(bf16_t* p, const float (&f)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(gdn::f32x2_to_bf16x2(f[0], f[1]), gdn::f32x2_to_bf16x2(f[2], f[3]));
}
__device__ __forceinline__ void put4(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// Where pair p stands.
struct Place {
    int a, b;
};
__device__ __forceinline__ Place place(int p, int rot, bool neighbours) {
    if (!neighbours && p < rot / 2) return {p, p + rot / 2};
    return {2 * p, 2 * p + 1};
}
// N pairs from p0 on: one pair, or four that are all halves or all neighbours
// (rot / 2 a multiple of 4) on whole vectors.
template <typename T, int N> __device__ __forceinline__ void load_pairs(const T* x, int p0, int rot, bool neighbours, float (&a)[N], float (&b)[N]) {
    if constexpr (N == 1) {
        const Place at = place(p0, rot, neighbours);
        a[0] = gdn::to_f32(x[at.a]);
        b[0] = gdn::to_f32(x[at.b]);
    } else if (!neighbours && p0 < rot / 2) {
        get4(x + p0, a);
        get4(x + p0 + rot / 2, b);
    } else {
        float u[4], v[4];
        get4(x + 2 * p0, u);
        get4(x + 2 * p0 + 4, v);
        a[0] = u[0]; b[0] = u[1]; a[1] = u[2]; b[1] = u[3];
        a[2] = v[0]; b[2] = v[1]; a[3] = v[2]; b[3] = v[3];
    }
}
template <typename T, int N> __device__ __forceinline__ void store_pairs(T* x, int p0, int rot, bool neighbours, const float (&a)[N], const float (&b)[N]) {
    if constexpr (N == 1) {
        const Place at = place(p0, rot, neighbours);
        x[at.a] = gdn::from_f32<T>(a[0]);
        x[at.b] = gdn::from_f32<T>(b[0]);
    } else if (!neighbours && p0 < rot / 2) {
        put4(x + p0, a);
        put4(x + p0 + rot / 2, b);
    } else {
        const float u[4] = {a[0], b[0], a[1], b[1]}, v[4] = {a[2], b[2], a[3], b[3]};
        put4(x + 2 * p0, u);
        put4(x + 2 * p0 + 4, v);
    }
}

// N: pairs a lane moves together; NI: how often, 16 N NI >= d / 2.
template <typename T, int N, int NI, bool BACK>
__global__ __launch_bounds__(kThreads) void k_rotate(const RotateArgs A, int rows_at_once) {
    __shared__ float2 s_turn[kRotRows][kMaxPairs];   // cosine, sine
    // The weights' gradients of q and k: fp32 over kTerms heads, fp64 from there on, so that the error does not grow
    // with the rows (over 2^20 rows of 8 heads 11 half steps, now below 4; 8, 16, 32 heads at a time take 434, 431,
    // 428 us forward and backward over 32768 rows of 48 heads of 128, fp32 throughout 423).
    constexpr int kTerms = 32, kValues = 2 * kLanes * N * NI;
    __shared__ double s_dw[2][BACK ? kHeadsAtOnce : 1][BACK ? kValues : 1];
    const int tid = threadIdx.x, lane = tid % kLanes, grp = tid / kLanes;
    const int np = A.d / 2, nr = A.rot / 2;
    const bool neighbours = A.neighbours != 0;
    const int heads = A.heads[0] + A.heads[1];
    float w[2][NI][N][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int p = (k * kLanes + lane) * N + j;
                const Place at = place(p, A.rot, neighbours);
                w[t][k][j][0] = A.w[t] && p < np ? A.w[t][at.a] : 1.0f;
                w[t][k][j][1] = A.w[t] && p < np ? A.w[t][at.b] : 1.0f;
            }
    float dw[2][NI][N][2] = {};
    int terms = 0;
    auto each_dw = [&](auto f) {  // this lane's places in s_dw
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < NI; ++k)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int p = (k * kLanes + lane) * N + j;
                    if (p >= np) continue;
                    const Place at = place(p, A.rot, neighbours);
                    f(s_dw[t][grp][at.a], dw[t][k][j][0]);
                    f(s_dw[t][grp][at.b], dw[t][k][j][1]);
                }
    };
    if constexpr (BACK) each_dw([](double& sum, float&) { sum = 0.0; });
    auto hand_over = [&]() {
        each_dw([](double& sum, float& v) {
            sum += (double)v;
            v = 0.0f;
        });
        terms = 0;
    };
    const float inv_over = 1.0f / A.over;

    for (int64_t r0 = (int64_t)blockIdx.x * rows_at_once; r0 < A.n_rows; r0 += (int64_t)gridDim.x * rows_at_once) {
        const int rows = (int)min((int64_t)rows_at_once, A.n_rows - r0);
        __syncthreads();  // the angles before these are used up
        for (int j = tid; j < rows * nr; j += kThreads) {
            const int r = j / nr, p = j - r * nr;
            const double turns = (double)A.pos[r0 + r] * (double)A.inv_freq[p] * 0.15915494309189535;
            float sn, cs;
            const double part = turns - rint(turns);
            const float near = (float)part, off = (float)(part - (double)near) * 6.2831853f;
            sincospif(2.0f * near, &sn, &cs);
            s_turn[r][p] = make_float2(fmaf(-off, sn, cs), fmaf(off, cs, sn));
        }
        __syncthreads();
        for (int u = grp; u < rows * heads; u += kHeadsAtOnce) {
            const int r = u / heads, hh = u - r * heads, t = hh < A.heads[0] ? 0 : 1, h = t ? hh - A.heads[0] : hh;
            const int64_t row = r0 + r;
            const T* x = static_cast<const T*>(t ? A.x[1] : A.x[0]) + row * (t ? A.x_stride[1] : A.x_stride[0]) + (int64_t)h * A.d;
            T* y = static_cast<T*>(t ? A.y[1] : A.y[0]) + row * (t ? A.y_stride[1] : A.y_stride[0]) + (int64_t)h * A.d;
            float a[NI][N], b[NI][N], da[NI][N], db[NI][N];
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const int p0 = (k * kLanes + lane) * N;
#pragma unroll
                for (int j = 0; j < N; ++j) a[k][j] = b[k][j] = da[k][j] = db[k][j] = 0.0f;
                if (p0 < np) load_pairs<T, N>(x, p0, A.rot, neighbours, a[k], b[k]);
            }
            if constexpr (BACK) {
                const T* dy = static_cast<const T*>(t ? A.dy[1] : A.dy[0]) + row * (t ? A.dy_stride[1] : A.dy_stride[0]) + (int64_t)h * A.d;
#pragma unroll
                for (int k = 0; k < NI; ++k) {
                    const int p0 = (k * kLanes + lane) * N;
                    if (p0 < np) load_pairs<T, N>(dy, p0, A.rot, neighbours, da[k], db[k]);
                }
            }
            float ss = 0.0f;
#pragma unroll
            for (int k = 0; k < NI; ++k)
#pragma unroll
                for (int j = 0; j < N; ++j) ss = fmaf(a[k][j], a[k][j], fmaf(b[k][j], b[k][j], ss));
            ss = reduce16(ss);
            float square = ss * inv_over + A.eps, unit = 1.0f;
            // squares beyond fp32's range (|x| from some 2^60 on, or up to 2^-46 and eps no larger): the head, all
            // sixteen lanes of it, is taken times a power of two, and its gradient once more in the end
            if (!(square >= 0x1p-100f && square < __builtin_inff())) {
                unit = square < 1.0f ? 0x1p100f : 0x1p-70f;
                ss = 0.0f;
#pragma unroll
                for (int k = 0; k < NI; ++k)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        a[k][j] *= unit;
                        b[k][j] *= unit;
                        ss = fmaf(a[k][j], a[k][j], fmaf(b[k][j], b[k][j], ss));
                    }
                square = reduce16(ss) * inv_over + A.eps * unit * unit;
            }
            const float root = 1.0f / sqrtf(square);
            if constexpr (!BACK) {
#pragma unroll
                for (int k = 0; k < NI; ++k) {
                    const int p0 = (k * kLanes + lane) * N;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float wa = t ? w[1][k][j][0] : w[0][k][j][0], wb = t ? w[1][k][j][1] : w[0][k][j][1];
                        const float na = a[k][j] * root * wa, nb = b[k][j] * root * wb;
                        a[k][j] = na;
                        b[k][j] = nb;
                        if (p0 + j < nr) {
                            const float2 c = s_turn[r][p0 + j];
                            a[k][j] = fmaf(na, c.x, -(nb * c.y));
                            b[k][j] = fmaf(nb, c.x, na * c.y);
                        }
                    }
                    if (p0 < np) store_pairs<T, N>(y, p0, A.rot, neighbours, a[k], b[k]);
                }
            } else {
                float along = 0.0f;
#pragma unroll
                for (int k = 0; k < NI; ++k) {
                    const int p0 = (k * kLanes + lane) * N;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float wa = t ? w[1][k][j][0] : w[0][k][j][0], wb = t ? w[1][k][j][1] : w[0][k][j][1];
                        float ga = da[k][j], gb = db[k][j];
                        if (p0 + j < nr) {
                            const float2 c = s_turn[r][p0 + j];
                            const float ta = fmaf(ga, c.x, gb * c.y), tb = fmaf(gb, c.x, -(ga * c.y));
                            ga = ta;
                            gb = tb;
                        }
                        const float ua = a[k][j] * root, ub = b[k][j] * root;
                        a[k][j] = ua;
                        b[k][j] = ub;
                        if (t) {
                            dw[1][k][j][0] = fmaf(ga, ua, dw[1][k][j][0]);
                            dw[1][k][j][1] = fmaf(gb, ub, dw[1][k][j][1]);
                        } else {
                            dw[0][k][j][0] = fmaf(ga, ua, dw[0][k][j][0]);
                            dw[0][k][j][1] = fmaf(gb, ub, dw[0][k][j][1]);
                        }
                        da[k][j] = ga * wa;
                        db[k][j] = gb * wb;
                        along = fmaf(da[k][j], ua, fmaf(db[k][j], ub, along));
                    }
                }
                along = reduce16(along) * inv_over;
#pragma unroll
                for (int k = 0; k < NI; ++k) {
                    const int p0 = (k * kLanes + lane) * N;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        da[k][j] = root * (da[k][j] - a[k][j] * along) * unit;
                        db[k][j] = root * (db[k][j] - b[k][j] * along) * unit;
                    }
                    if (p0 < np) store_pairs<T, N>(y, p0, A.rot, neighbours, da[k], db[k]);
                }
                if (A.part && ++terms == kTerms) hand_over();
            }
        }
    }
    if constexpr (BACK) {
        if (!A.part) return;
        hand_over();
        __syncthreads();
        for (int e = tid; e < 2 * A.d; e += kThreads) {
            const int t = e / A.d;
            double sum = 0.0;
            for (int q = 0; q < kHeadsAtOnce; ++q) sum += s_dw[t][q][e - t * A.d];
            A.part[(int64_t)blockIdx.x * 2 * A.d + e] = sum;
        }
    }
}

// dw[t][e] = the sum over the workgroups, in 64 bits and a fixed order.
__global__ __launch_bounds__(kThreads) void k_rotate_sum(const double* part, int64_t groups, int32_t d, float* dwq, float* dwk) {
    __shared__ double s_part[kThreads];
    const int e = blockIdx.x, t = blockIdx.y, tid = threadIdx.x;
    float* const out = t ? dwk : dwq;
    if (!out) return;
    double sum = 0.0;
    for (int64_t b = tid; b < groups; b += kThreads) sum += part[(b * 2 + t) * d + e];
    s_part[tid] = sum;
    __syncthreads();
    for (int n = kThreads / 2; n > 0; n >>= 1) {
        if (tid < n) s_part[tid] += s_part[tid + n];
        __syncthreads();
    }
    if (tid == 0) out[e] = (float)s_part[0];
}

int64_t rotate_groups(int64_t n_rows) { return n_rows < 1024 ? n_rows : 1024; }

template <typename T, int N, int NI> hipError_t run_rotate(const RotateArgs& a, bool back, hipStream_t s) {
    if (back) {
        const int64_t groups = rotate_groups(a.n_rows);
        const int rows = groups * kRotRows <= a.n_rows ? kRotRows : 1;
        if (groups > 0) hipLaunchKernelGGL((k_rotate<T, N, NI, true>), dim3((unsigned)groups), dim3(kThreads), 0, s, a, rows);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || (!a.dw[0] && !a.dw[1])) return e;
        hipLaunchKernelGGL(k_rotate_sum, dim3((unsigned)a.d, 2), dim3(kThreads), 0, s, a.part, groups, a.d, a.dw[0], a.dw[1]);
        return hipGetLastError();
    }
    const int rows = a.n_rows >= 4096 ? kRotRows : 1;
    int64_t groups = (a.n_rows + rows - 1) / rows;
    if (groups > 8192) groups = 8192;
    if (groups > 0) hipLaunchKernelGGL((k_rotate<T, N, NI, false>), dim3((unsigned)groups), dim3(kThreads), 0, s, a, rows);
    return hipGetLastError();
}
template <typename T> hipError_t pick_rotate(const RotateArgs& a, bool back, hipStream_t s) {
    const int np = a.d / 2;
    if (a.vec) return np <= 4 * kLanes ? run_rotate<T, 4, 1>(a, back, s) : run_rotate<T, 4, 2>(a, back, s);
    if (np <= 2 * kLanes) return run_rotate<T, 1, 2>(a, back, s);
    return np <= 4 * kLanes ? run_rotate<T, 1, 4>(a, back, s) : run_rotate<T, 1, 8>(a, back, s);
}
hipError_t launch_rotate(const RotateArgs& a, bool back, hipStream_t s) {
    return a.bf16 ? pick_rotate<bf16_t>(a, back, s) : pick_rotate<float>(a, back, s);
}

}  // namespace gdnl
