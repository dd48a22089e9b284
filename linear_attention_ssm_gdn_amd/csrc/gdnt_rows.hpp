// gdnt_rows.hpp -- rows as the scan kernels hold them: two channels a lane,
// the rows of one tensor that a wave works on, blocks of the 8-bit checkpoint.
#pragma once

#include "gdnt_device.hpp"

namespace gdnt {

constexpr int FR = GDNT_CKPT_ROWS;  // consecutive rows of a lane: 16

// Two channels of a row as they are stored.
template <typename T> struct Raw2;
template <> struct Raw2<bf16_t> {
    uint32_t v;
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
    // the larger of |value|s as bits, kept per channel; NaN above Inf above all others
    __device__ __forceinline__ uint32_t top(uint32_t t) const {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, t),
                                                                     __builtin_bit_cast(u16x2, v & 0x7fff7fffu)));
    }
    static __device__ __forceinline__ uint32_t top_bits(uint32_t t) {
        const uint32_t a = t << 16, b = t & 0xffff0000u;
        return a > b ? a : b;
    }
};
template <> struct Raw2<float> {
    float2 v;
    __device__ __forceinline__ float get(int i) const { return i ? v.y : v.x; }
    __device__ __forceinline__ uint32_t top(uint32_t t) const {
        const uint32_t a = __float_as_uint(v.x) & 0x7fffffffu, b = __float_as_uint(v.y) & 0x7fffffffu;
        return max(t, max(a, b));
    }
    static __device__ __forceinline__ uint32_t top_bits(uint32_t t) { return t; }
};
template <typename T> __device__ __forceinline__ Raw2<T> zero2() {
    Raw2<T> r;
    __builtin_memset(&r, 0, sizeof(r));
    return r;
}
// The rows of one tensor that a wave works on.  `first`: the wave's first row,
// `col` its first channel, `lane_at` the lane's own first element from there;
// row r of the lane is r rows further down.  A buffer descriptor makes a row's
// place a scalar offset and a lane's place one vector register for all rows
// (32 bits: row strides end at 2^24 elements); it ends with the tensor.
// PAIR: a lane's two channels move together, wherever the row starts, for bf16
// at odd offsets as dwords across dword boundaries (forward and backward over
// 16692 rows take 596 us with 4095 bf16 channels, 571 with 4094; channel by
// channel it was 1146).  Else there is only one channel.  The lane with an odd
// count's last channel loads a pair all the same, with what is behind it (the
// descriptor's end, or what fills the row); last_alone then loads that channel
// alone, in the one column that has it.  ODD false: the count is even, no lane
// has one channel alone.
template <typename T, bool PAIR, bool ODD = true> struct WaveRows {
    static_assert(PAIR || ODD, "one channel is an odd count");
    __amdgpu_buffer_rsrc_t rs;
    uint32_t row, at;  // bytes
    bool odd;          // uniform: a lane here has one channel
    __device__ __forceinline__ WaveRows(const void* base, int64_t stride, int64_t n_rows, int64_t first, int32_t C,
                                        int64_t col, int64_t lane_at)
        : row((uint32_t)stride * (uint32_t)sizeof(T)), at((uint32_t)lane_at * (uint32_t)sizeof(T)),
          odd(ODD && (C & 1) && C - col < 128) {
        // where rows are walked tile after tile, keeps the rows' offsets from being held in registers
        asm volatile("" : "+s"(row));
        int64_t bytes = ((n_rows - 1 - first) * stride + C - col) * (int64_t)sizeof(T);
        bytes = bytes < 0 ? 0 : bytes > 0xfffffffcll ? 0xfffffffcll : bytes;
        rs = __builtin_amdgcn_make_buffer_rsrc(static_cast<T*>(const_cast<void*>(base)) + first * stride + col, 0,
                                               (uint32_t)bytes, 0x00020000);
    }
    __device__ __forceinline__ Raw2<T> load(int r) const {
        Raw2<T> v;
        if constexpr (!PAIR) v = load_one(r);
        else if constexpr (sizeof(T) == 2) v.v = __builtin_amdgcn_raw_buffer_load_b32(rs, at, r * row, 0);
        else v.v = __builtin_bit_cast(float2, __builtin_amdgcn_raw_buffer_load_b64(rs, at, r * row, 0));
        return v;
    }
    __device__ __forceinline__ Raw2<T> load_one(int r) const {
        Raw2<T> v;
        if constexpr (sizeof(T) == 2) v.v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, at, r * row, 0);
        else v.v = make_float2(__uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, at, r * row, 0)), 0.0f);
        return v;
    }
    // rows: those of the lane that belong to a sequence, as bits
    __device__ __forceinline__ void last_alone(Raw2<T> (&v)[FR], uint32_t rows, int nc) const {
        if (!PAIR || !ODD || !odd || nc != 1) return;
#pragma unroll
        for (int r = 0; r < FR; ++r)
            if (rows >> r & 1u) v[r] = load_one(r);
        // nothing left under way: where the ways join, waits count the first loads only
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    }
    __device__ __forceinline__ void store(int r, int nc, float a, float b) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t v = gdn::f32x2_to_bf16x2(a, b);
            if (PAIR && nc == 2) __builtin_amdgcn_raw_buffer_store_b32(v, rs, at, r * row, 0);
            if (ODD && odd && nc == 1) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)v, rs, at, r * row, 0);
        } else {
            const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            if (PAIR && nc == 2) __builtin_amdgcn_raw_buffer_store_b64((u32x2){x, y}, rs, at, r * row, 0);
            if (ODD && odd && nc == 1) __builtin_amdgcn_raw_buffer_store_b32(x, rs, at, r * row, 0);
        }
    }
};

// A block of the checkpoint (16 rows by 4 channels) is two neighbouring
// lanes' values; each lane writes and reads eight whole rows of it (32 of its
// 64 bytes), the even lane the upper ones.  swap_halves turns between the two
// views: w[r] as bytes {row r: c0 c1, row r + 8: c0 c1} of the lane's two
// channels, and w[r] as the four channels of one row.  It is its own inverse.
__device__ __forceinline__ uint32_t swap_halves(uint32_t w, int lane) {
    const uint32_t x = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0xB1, 0xF, 0xF, false);
    return (lane & 1) ? __builtin_amdgcn_perm(w, x, 0x07060302u) : __builtin_amdgcn_perm(x, w, 0x05040100u);
}

}  // namespace gdnt
