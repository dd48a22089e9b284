// gdnl_cache.hip -- state pages into 8-bit entries and back.
//
// Sixteen lanes hold a block of 64 columns of a row, four columns each, so a
// block's largest value is one maximum over a DPP row; a workgroup takes 16
// blocks at a time, four times.  v * fl(127/m) + 1.5 2^23 in one fused
// multiply-add rounds once to an integer, which then is the low byte.  Bound by
// the pages' bytes: 96 pages of 32 heads of 128 x 128 in fp32 take 62 us into entries
// (4.1 TB/s) and 39 us back (6.5 TB/s, the entries just written still near).
#include "gdn_device.hpp"
#include "gdnl_kernels.h"
#include "gdnt_device.hpp"

namespace gdnl {

using gdn::bf16_t;
using gdnt::raise;

constexpr int kBlocksMine = 4;                         // blocks of a thread, one behind the other
constexpr int kBlocks = kThreads / 16 * kBlocksMine;   // of a workgroup
// The largest scale whose 127-fold is finite: that of a block around the
// largest fp32 number is one step above it.
constexpr float kTopScale = 0x1.020406p+121f;

__device__ __forceinline__ uint32_t max16(uint32_t v) {
    auto other = [](uint32_t x, int c) {
        switch (c) {
            case 0: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false);
            case 1: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false);
            case 2: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false);
            default: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, false);
        }
    };
    v = max(v, other(v, 0));
    v = max(v, other(v, 1));
    v = max(v, other(v, 2));
    return max(v, other(v, 3));
}

template <typename S, bool VEC, bool STORE>
__global__ __launch_bounds__(kThreads) void k_cache(const CacheArgs A, int groups) {
    const int i = (int)(blockIdx.x / groups), tid = threadIdx.x, l = tid & 15;
    const int page = A.page[i], entry = A.entry[i];
    if (page < 0 || entry < 0) return;
    if (page >= A.n_pages || entry >= A.n_entries) {
        if (blockIdx.x % groups == 0 && tid == 0)
            raise(A.err, (page >= A.n_pages ? GDN_DEVERR_PAGE : 0u) | (entry >= A.n_entries ? GDN_DEVERR_CACHE : 0u));
        return;
    }
    const int per = (A.dv + 63) / 64;  // blocks of a row
    const int64_t n_blocks = A.rows * per, first = (int64_t)(blockIdx.x % groups) * kBlocks + (tid >> 4);
    S* st = static_cast<S*>(A.st) + (int64_t)page * A.st_stride;
    int8_t* q = A.q + (int64_t)entry * A.rows * A.dv;
    float* scale = A.scale + (int64_t)entry * n_blocks;
    int64_t at[kBlocksMine];
    int nc[kBlocksMine];
#pragma unroll
    for (int j = 0; j < kBlocksMine; ++j) {
        const int64_t b = first + j * (kThreads / 16), row = b / per;
        const int c = (int)(b - row * per) * 64 + 4 * l;
        at[j] = row * A.dv + c;
        nc[j] = b < n_blocks ? min(4, A.dv - c) : 0;
    }
    if constexpr (STORE) {
        gdnt::Raw4<S> v[kBlocksMine];
#pragma unroll
        for (int j = 0; j < kBlocksMine; ++j) {
            v[j] = gdnt::zero4<S>();
            if (nc[j] > 0) v[j] = gdnt::load4<S, VEC>(st + at[j], nc[j]);
        }
#pragma unroll
        for (int j = 0; j < kBlocksMine; ++j) {
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(v[j].get(k)) & 0x7fffffffu);
            top = max16(top);
            const float m = __uint_as_float(top);
            const bool finite = top < 0x7f800000u, live = finite && m >= 0x1p-100f;
            const float up = live ? 127.0f / m : 0.0f;
            const float sc = !finite ? __uint_as_float(0x7fc00000u) : live ? fminf(m / 127.0f, kTopScale) : 0.0f;
            uint32_t e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                e[k] = live ? __float_as_uint(fmaf(v[j].get(k), up, 12582912.0f)) & 0xffu : 0u;
            const uint32_t w = e[0] | (e[1] << 8) | (e[2] << 16) | (e[3] << 24);
            if (nc[j] > 0) {
                if (VEC) {
                    *reinterpret_cast<uint32_t*>(q + at[j]) = w;
                } else {
                    for (int k = 0; k < nc[j]; ++k) q[at[j] + k] = (int8_t)(w >> (8 * k));
                }
                if (l == 0) scale[first + j * (kThreads / 16)] = sc;
            }
        }
    } else {
        uint32_t w[kBlocksMine];
        float sc[kBlocksMine];
#pragma unroll
        for (int j = 0; j < kBlocksMine; ++j) {
            w[j] = 0;
            sc[j] = 0.0f;
            if (nc[j] > 0) {
                if (VEC) {
                    w[j] = *reinterpret_cast<const uint32_t*>(q + at[j]);
                } else {
                    for (int k = 0; k < nc[j]; ++k) w[j] |= (uint32_t)(uint8_t)q[at[j] + k] << (8 * k);
                }
                sc[j] = scale[first + j * (kThreads / 16)];
            }
        }
#pragma unroll
        for (int j = 0; j < kBlocksMine; ++j) {
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = (float)(int8_t)(w[j] >> (8 * k)) * sc[j];
            if (nc[j] > 0) gdnt::store4<VEC>(st + at[j], f, nc[j]);
        }
    }
}

template <typename S> hipError_t run_cache(const CacheArgs& a, bool store, hipStream_t s) {
    const int64_t blocks = a.rows * ((a.dv + 63) / 64), groups = (blocks + kBlocks - 1) / kBlocks;
    const dim3 grid((unsigned)(groups * a.n)), block(kThreads);
    if (store) {
        if (a.vec) hipLaunchKernelGGL((k_cache<S, true, true>), grid, block, 0, s, a, (int)groups);
        else hipLaunchKernelGGL((k_cache<S, false, true>), grid, block, 0, s, a, (int)groups);
    } else {
        if (a.vec) hipLaunchKernelGGL((k_cache<S, true, false>), grid, block, 0, s, a, (int)groups);
        else hipLaunchKernelGGL((k_cache<S, false, false>), grid, block, 0, s, a, (int)groups);
    }
    return hipGetLastError();
}
hipError_t launch_cache(const CacheArgs& a, bool store, hipStream_t s) {
    return a.bf16 ? run_cache<bf16_t>(a, store, s) : run_cache<float>(a, store, s);
}

}  // namespace gdnl
