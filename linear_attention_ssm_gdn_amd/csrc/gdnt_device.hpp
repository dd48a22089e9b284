// gdnt_device.hpp -- device helpers of the training-side operators: rows of
// four channels, the row map, the gates of the vector-state recurrence.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_device.hpp"
#include "gdnt_kernels.h"
#include "../../include/gdn_train.h"

namespace gdnt {

using gdn::bf16_t;
using gdn::from_f32;
using gdn::to_f32;

// Four channels of a row as they are stored.
template <typename T> struct Raw4;
template <> struct Raw4<bf16_t> {
    uint2 v;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = (i & 2) ? v.y : v.x;
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ __forceinline__ void set(int i, bf16_t e) {
        uint32_t& w = (i & 2) ? v.y : v.x;
        w = (i & 1) ? ((w & 0xffffu) | ((uint32_t)e << 16)) : ((w & 0xffff0000u) | e);
    }
};
template <> struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ float get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
    __device__ __forceinline__ void set(int i, float e) { (i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w) = e; }
};

template <typename T> __device__ __forceinline__ Raw4<T> zero4() {
    Raw4<T> r;
    __builtin_memset(&r, 0, sizeof(r));
    return r;
}

// p: the first of the four channels; nc: how many of them exist.  VEC: four,
// and p on a vector's boundary; else p on an element's.
template <typename T, bool VEC> __device__ __forceinline__ Raw4<T> load4(const T* p, int nc) {
    Raw4<T> r = zero4<T>();
    if constexpr (VEC) {
        r.v = *reinterpret_cast<const decltype(r.v)*>(p);
    } else if (nc == 4) {
        __builtin_memcpy(&r.v, p, sizeof(r.v));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < nc) r.set(i, p[i]);
    }
    return r;
}
template <bool VEC> __device__ __forceinline__ void store4(bf16_t* p, const float (&f)[4], int nc) {
    if constexpr (VEC) {
        *reinterpret_cast<uint2*>(p) = make_uint2(gdn::f32x2_to_bf16x2(f[0], f[1]), gdn::f32x2_to_bf16x2(f[2], f[3]));
    } else if (nc == 4) {
        const uint2 v = make_uint2(gdn::f32x2_to_bf16x2(f[0], f[1]), gdn::f32x2_to_bf16x2(f[2], f[3]));
        __builtin_memcpy(p, &v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < nc) p[i] = from_f32<bf16_t>(f[i]);
    }
}
template <bool VEC> __device__ __forceinline__ void store4(float* p, const float (&f)[4], int nc) {
    if constexpr (VEC) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else if (nc == 4) {
        const float4 v = make_float4(f[0], f[1], f[2], f[3]);
        __builtin_memcpy(p, &v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < nc) p[i] = f[i];
    }
}

// State pages and per-sequence gradients: touched once per sequence, so one
// value at a time serves.
__device__ __forceinline__ float load_state(const void* base, int64_t at, int32_t dtype) {
    return dtype == GDN_BF16 ? to_f32(static_cast<const bf16_t*>(base)[at]) : static_cast<const float*>(base)[at];
}
__device__ __forceinline__ void store_state(void* base, int64_t at, int32_t dtype, float v) {
    if (dtype == GDN_BF16) static_cast<bf16_t*>(base)[at] = from_f32<bf16_t>(v);
    else static_cast<float*>(base)[at] = v;
}

__device__ __forceinline__ void raise(int32_t* err, uint32_t bit) {
    if (err) atomicOr(reinterpret_cast<unsigned int*>(err), bit);
}

// Bounds of a sequence are in range and not decreasing.
__device__ __forceinline__ bool bounds_ok(int64_t n_rows, int c0, int c1) {
    return c0 >= 0 && c1 >= c0 && (int64_t)c1 <= n_rows;
}
// Is sequence s valid, given that some sequence has bad bounds?  It may not
// begin before the end of a valid one above it, so every row has one owner.
__device__ inline bool valid_slow(const int32_t* cu, int64_t n_rows, int s) {
    int end = 0;
    for (int j = 0; j <= s; ++j) {
        const int c0 = cu[j], c1 = cu[j + 1];
        const bool ok = c0 >= end && bounds_ok(n_rows, c0, c1);
        if (j == s) return ok;
        if (ok) end = c1;
    }
    return false;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTiny = 1.17549435e-38f;  // smallest normal number

__device__ __forceinline__ float rcp(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }

// softplus(z) = max(z, 0) + log1p(t), t = e^{-|z|} in [0, 1], and log1p(t) =
// t p(t) with p the interpolation of log1p(t) / t of degree 8 at the
// Chebyshev nodes of [0, 1] (3.4e-8 off, 1.7e-7 with fp32's roundings).
// Relative accuracy holds for small softplus too, where log(1 + t) would
// lose it: a decay near 1 is raised to long powers.
// max(z, 0) ends at 2^100, where e^g is long 0 and g = -exp(A_log) softplus(z)
// still a number: the sum of dg g takes 0 times it.  (A median of three costs
// what a maximum does; a NaN z is in t.)
// The coefficients sit in scalar registers: a vector instruction takes one
// such operand for free, while a literal costs a move into the accumulator.
template <uint32_t BITS> __device__ __forceinline__ float scalar_const() {
    float c;
    asm("s_mov_b32 %0, %1" : "=s"(c) : "i"(BITS));
    return c;
}
struct SoftplusC {
    float c[9], top;
};
__device__ __forceinline__ SoftplusC softplus_consts() {
    SoftplusC k;
    k.c[8] = scalar_const<0x3ba7f8ddu>();  // 0.00512610236f
    k.c[7] = scalar_const<0xbcee2cbcu>();  // -0.0290740654f
    k.c[6] = scalar_const<0x3d9ec0c1u>();  // 0.0775160864f
    k.c[5] = scalar_const<0xbe0b497au>();  // -0.136022478f
    k.c[4] = scalar_const<0x3e4358e6u>();  // 0.190768808f
    k.c[3] = scalar_const<0xbe7e5082u>();  // -0.248353988f
    k.c[2] = scalar_const<0x3eaa96bau>();  // 0.333181202f
    k.c[1] = scalar_const<0xbeffff46u>();  // -0.499994457f
    k.c[0] = scalar_const<0x3f7fffffu>();  // 0.99999994f
    // 2^100, in a vector register: one more scalar is spilled in the backward
    // pass (forward + backward over 32768 x 4096 in bf16: 751 us, 745 so)
    asm("v_mov_b32 %0, 0x71800000" : "=v"(k.top));
    return k;
}
__device__ __forceinline__ float softplus_t(const SoftplusC& k, float z, float& t) {
    t = exp2_hw(-fabsf(z) * kLog2e);
    float p = k.c[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) p = fmaf(t, p, k.c[i]);
    return fmaf(t, p, __builtin_amdgcn_fmed3f(z, 0.0f, k.top));
}
// sigmoid(b); the hardware exponential and reciprocal, about an ulp each.
__device__ __forceinline__ float sigmoid_hw(float b) { return rcp(1.0f + exp2_hw(-b * kLog2e)); }

// Per-channel constants: dt_bias and -exp(A_log) log2(e), so that
// e^{g} = 2^{k softplus(z)}.
struct ChanP {
    float dt[4], k[4];
};
__device__ __forceinline__ ChanP load_params(const float* a_log, const float* dt_bias, int64_t c0, int nc) {
    ChanP p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p.dt[i] = i < nc ? dt_bias[c0 + i] : 0.0f;
        p.k[i] = i < nc ? -expf(a_log[c0 + i]) * kLog2e : 0.0f;
    }
    return p;
}

}  // namespace gdnt
