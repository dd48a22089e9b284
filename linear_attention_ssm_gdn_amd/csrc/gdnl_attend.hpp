// gdnl_attend.hpp -- linear attention over chunks of 64 rows on matrix cores,
// forward or backward in time (AttendArgs), for one act type.
//
// A workgroup walks a segment's chunks for one value head; each of its four or
// eight waves owns 16 NT columns of the head's state S, all DK rows of them, in
// the accumulators, so S never leaves the registers.  Matrix products reduce over
// 32 positions at a time, eight to a lane, and which positions a lane holds is
// free as long as both operands agree.  The choice here, 4g..4g+3 of two tiles
// of 16 (g = lane / 16), is how a product leaves its rows in the accumulators:
//   - S serves as the right operand of q S without an exchange between lanes;
//   - k q^T leaves (q k^T) as the left operand of P v, through LDS once, since
//     every wave needs all of it.
// v, and k for the state's update, are read from row-major LDS tiles by
// transposing loads (fp32: value by value), one reading of v serving P v and
// the update.
//
// Decays.  G is summed within a chunk in 64 bits and kept as two floats
// (decays_of, once for all passes), so e^{G_x - G_y} is good to the difference's
// own digits; it is set, not multiplied, to zero where y lies ahead of x.
//
// Roundings with bf16 rows.  The products of q, k and v themselves are exact.
// What is not a bf16 number (P, S, the decayed rows of the state's update) is
// split into three terms of eight bits, which leave nothing: states are as good
// as their fp32 sums, outputs as these rounded once.
//
// What bounds it: vector and matrix instructions, on units of their own, and waits
// between them.  Over 4 x 8192 rows of 32 heads of 128 x 128 in bf16 the outputs take
// 320-345 us, some 650 vector and 119 matrix instructions a wave and chunk, busy 66%
// and 41% of the time; the 0.9 GB would take 175 us at a copy's rate.  fp32 rows are bound by the matrix instructions (68% busy, 85 TFLOP/s over
// 16384 rows).  Why eight waves of 16 columns: two workgroups then fit a compute
// unit's registers (128 a lane) and LDS, and one computes while the other waits at
// a barrier; four waves of 32 columns were no faster.  Chunks of 64 rows: with 32
// the work on the state would come twice as often, with 128 two workgroups would
// not fit LDS.
#pragma once

#include "gdn_device.hpp"
#include "gdnl_kernels.h"

namespace gdnl {

using gdn::bf16_t;
using gdn::lds_barrier;
using gdn::reduce16;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kTri = 10;  // tiles of 16 x 16 on or below the diagonal of 64 x 64

__device__ __forceinline__ int tri(int lo, int hi) { return hi * (hi + 1) / 2 + lo; }
// P in LDS: for an output tile x, the source tiles 2 ys and 2 ys + 1 side by
// side, as one operand of a product takes them; six such pairs have a tile on
// the right side of the diagonal.  Two of them have one alone, which stands by
// itself, the other half of the operand being zeros.
template <bool BACK> __host__ __device__ constexpr bool is_pair(int x, int ys) { return BACK ? 2 * ys + 1 >= x : 2 * ys <= x; }
template <bool BACK> __host__ __device__ constexpr bool is_alone(int x, int ys) { return x == 2 * ys + (BACK ? 1 : 0); }
// In tiles, where a pair stands among the ten.
template <bool BACK> __host__ __device__ constexpr int pair(int x, int ys) {
    // forward (0,0) (1,0) (2,0) (2,1) (3,0) (3,1), backward (0,0) (0,1) (1,0) (1,1) (2,1) (3,1)
    return BACK ? 0x975420 >> 4 * (x < 2 ? 2 * x + ys : x + 2) & 15 : 0x865310 >> 4 * (x < 2 ? x : 2 * x - 2 + ys) & 15;
}

__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }

// Vector instructions read a product's result late enough (32 wait states: see
// gdn_chunked.hip).
template <int N> __device__ __forceinline__ void settle(f32x4 (&a)[N]) {
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(a[i]));
}

// Eight positions of one operand row or column.
template <typename T> struct Frag;
template <> struct Frag<bf16_t> { u32x4 v; };
template <> struct Frag<float> { float v[8]; };

__device__ __forceinline__ f32x4 mma(const Frag<bf16_t>& a, const Frag<bf16_t>& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c,
                                                   0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
}

// The same in two chains: a matrix instruction of fp32 rounds after each of its
// products, so shorter chains are the more exact.
__device__ __forceinline__ void mma_chains(const Frag<float>& a, const Frag<float>& b, f32x4 (&c)[2]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c[e & 1], 0, 0, 0);
}

// x as a sum of bf16 terms: the leading eight bits cut off, so that what is
// left is exact, the last term rounded.
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float leading(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
template <int TERMS> __device__ __forceinline__ void split2(float a, float b, uint32_t (&t)[TERMS]) {
#pragma unroll
    for (int i = 0; i < TERMS - 1; ++i) {
        t[i] = high_halves(a, b);
        a -= leading(a);
        b -= leading(b);
    }
    t[TERMS - 1] = gdn::f32x2_to_bf16x2(a, b);
}
template <int TERMS> __device__ __forceinline__ void split(const float (&f)[8], Frag<bf16_t> (&t)[TERMS]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[TERMS];
        split2<TERMS>(f[2 * i], f[2 * i + 1], w);
#pragma unroll
        for (int j = 0; j < TERMS; ++j) t[j].v[i] = w[j];
    }
}
template <int TERMS> __device__ __forceinline__ void split(const float (&f)[8], Frag<float> (&t)[TERMS]) {
    static_assert(TERMS == 1, "fp32 is one term");
#pragma unroll
    for (int i = 0; i < 8; ++i) t[0].v[i] = f[i];
}
__device__ __forceinline__ void values(const Frag<bf16_t>& t, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(t.v[i] << 16);
        f[2 * i + 1] = __uint_as_float(t.v[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void values(const Frag<float>& t, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = t.v[i];
}

// 64 rows of W values, row-major in pieces of 16 bytes whose place within the
// row is exclusive-ored by the row: all the readings below spread over all
// banks, and what the row contributes is the same for rows 16 apart, so that a
// lane needs few addresses, the rest being constants of the instructions.
template <typename T, int W> struct Tile {
    static constexpr int kPieces = W * (int)sizeof(T) / 16;           // of a row
    static constexpr int kElems = 16 / (int)sizeof(T);
    static constexpr int kRow = W * (int)sizeof(T);
    static constexpr int kBytes = kChunk * kRow;
    static __device__ __forceinline__ int place(int row, int piece) {
        // bf16: sixteen rows, a piece each, and eight rows, two pieces each, are both read at once
        const int r = W == 128 ? row : row >> 1;
        const int x = sizeof(T) == 4 ? (row & 15) : W == 128 ? (r & 7) << 1 | (r >> 3 & 1) : (r & 3) << 1 | (r >> 2 & 1);
        return row * kRow + ((piece ^ x) << 4);
    }
    // Positions 4g..4g+3 of the 16s at 32 ks and 32 ks + 16, of row 16 b + i.
    // `base`: row_base(); what ks adds to a lane's piece is exclusive-ored too.
    static __device__ __forceinline__ int row_base(int g, int i) {
        return sizeof(T) == 2 ? place(i, g >> 1) + (g & 1) * 8 : place(i, g);
    }
    static __device__ __forceinline__ Frag<T> by_row(const char* t, int base, int b, int ks) {
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            const char* const p = t + b * 16 * kRow;
            const u32x2 a = *reinterpret_cast<const u32x2*>(p + (base ^ (4 * ks) << 4));
            const u32x2 c = *reinterpret_cast<const u32x2*>(p + (base ^ (4 * ks + 2) << 4));
            f.v = u32x4{a.x, a.y, c.x, c.y};
        } else {
            const char* const p = t + b * 16 * kRow + (ks >> 1) * 256;
            const f32x4 a = *reinterpret_cast<const f32x4*>(p + (base ^ (8 * (ks & 1)) << 4));
            const f32x4 c = *reinterpret_cast<const f32x4*>(p + (base ^ (8 * (ks & 1) + 4) << 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f.v[e] = a[e];
                f.v[4 + e] = c[e];
            }
        }
        return f;
    }
    // Rows 4g..4g+3 of the 16s at 32 ys and 32 ys + 16, of column 16 m + i.
    // bf16: lanes 4j..4j+3 of a group of 16 name row 4g + j, 16 columns of it;
    // the transposing load gives each lane a column.
    static __device__ __forceinline__ int col_base(int g, int i) {
        return sizeof(T) == 2 ? place(4 * g + (i >> 2), (i & 3) >> 1) + (i & 1) * 8
                              : 4 * g * kRow + (((i >> 2) ^ (4 * g)) << 4) + (i & 3) * 4;
    }
    static __device__ __forceinline__ Frag<T> by_col(const char* t, int base, int ys, int m) {
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const char* const p = t + ys * 32 * kRow + (base ^ (2 * m) << 4);
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * kRow));
            const u32x2 a2 = __builtin_bit_cast(u32x2, a), b2 = __builtin_bit_cast(u32x2, b);
            f.v = u32x4{a2.x, a2.y, b2.x, b2.y};
        } else {
            const char* const p = t + ys * 32 * kRow + (m >> 2) * 256;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f.v[e] = *reinterpret_cast<const float*>(p + ((e >> 2) * 16 + (e & 3)) * kRow + (base ^ (4 * (m & 3) + (e & 3)) << 4));
        }
        return f;
    }
    // The same reading from a tile that is read by rows alone (put_by_row): a
    // lane's eight bf16 positions stand together.
    static __device__ __forceinline__ int whole_base(int g, int i) {
        return sizeof(T) == 2 ? i * kRow + ((g ^ (i & (kPieces - 1))) << 4) : row_base(g, i);
    }
    static __device__ __forceinline__ Frag<T> whole(const char* t, int base, int b, int ks) {
        if constexpr (sizeof(T) == 2) {
            Frag<T> f;
            f.v = *reinterpret_cast<const u32x4*>(t + b * 16 * kRow + (base ^ (4 * ks) << 4));
            return f;
        } else {
            return by_row(t, base, b, ks);
        }
    }
    // Where four bf16 columns from 4 q on stand in such a tile.
    static __device__ __forceinline__ int quad(int row, int q) {
        return row * kRow + (((q >> 3) * 4 + (q & 3)) ^ (row & (kPieces - 1))) * 16 + (q >> 2 & 1) * 8;
    }
    static __device__ __forceinline__ void put_by_row(char* t, int row, int piece, u32x4 v) {
        if constexpr (sizeof(T) == 2) {
            // columns 8 piece..: quads 2 (piece & 1) and the next of the first or second 16 of 32
            const int to = quad(row, 2 * piece);
            *reinterpret_cast<u32x2*>(t + to) = u32x2{v.x, v.y};
            *reinterpret_cast<u32x2*>(t + (to ^ 16)) = u32x2{v.z, v.w};
        } else {
            *reinterpret_cast<u32x4*>(t + place(row, piece)) = v;
        }
    }
    static __device__ __forceinline__ T* at(char* t, int row, int c) {
        return reinterpret_cast<T*>(t + place(row, c / kElems)) + c % kElems;
    }
};

template <typename T> __device__ __forceinline__ bool not_finite(T v);
template <> __device__ __forceinline__ bool not_finite<bf16_t>(bf16_t v) { return (v & 0x7f80u) == 0x7f80u; }
template <> __device__ __forceinline__ bool not_finite<float>(float v) {
    return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u;
}
// Some value of the piece is not finite.
template <typename T> __device__ __forceinline__ bool piece_not_finite(u32x4 w) {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) any |= ((w[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        else any |= ((w[i] & 0x7f800000u) + 0x00800000u) & 0x80000000u;
    }
    return any != 0;
}

// A buffer descriptor of the first n rows of a chunk (none for n <= 0): a read
// beyond is 0, a write beyond is dropped, without a branch.  Rows begin within
// 32 bits of the first (row strides end at 2^24 elements); kNowhere is beyond
// every descriptor.
constexpr uint32_t kNowhere = 0xffffff00u;
template <typename T> __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const void* p, int64_t stride, int64_t row0, int64_t at, int n, int d) {
    const uint32_t bytes = n > 0 ? ((uint32_t)(n - 1) * (uint32_t)stride + (uint32_t)d) * (uint32_t)sizeof(T) : 0u;
    return __builtin_amdgcn_make_buffer_rsrc(static_cast<T*>(const_cast<void*>(p)) + row0 * stride + at, 0, bytes, 0x00020000);
}

// A thread's pieces of 64 rows of a head, on their way to LDS.  Rows from n on
// and columns from d on are zeros.
template <typename T, int W, int THREADS, bool VEC> struct Fetch {
    using L = Tile<T, W>;
    static constexpr int kMine = kChunk * L::kPieces / THREADS, kStep = THREADS / L::kPieces;  // kStep rows between two
    u32x4 r[kMine];
    __device__ __forceinline__ void load(const Rows& R, int head, int d, int64_t row0, int n, int tid) {
        const __amdgpu_buffer_rsrc_t rs = rows_buffer<T>(R.p, R.stride, row0, (int64_t)(head / R.per) * d, n, d);
        const int row = tid / L::kPieces, c = tid % L::kPieces * L::kElems;
        const bool some = VEC ? c < d : true;
        uint32_t off = some ? ((uint32_t)row * (uint32_t)R.stride + (uint32_t)c) * (uint32_t)sizeof(T) : kNowhere;
        const uint32_t step = some ? kStep * (uint32_t)R.stride * (uint32_t)sizeof(T) : 0u;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            if constexpr (VEC) {
                r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
            } else {
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < L::kElems; ++e) {
                    const bool in = c + e < d;
                    const uint32_t at = in ? off + e * (uint32_t)sizeof(T) : kNowhere;
                    if constexpr (sizeof(T) == 2) w[e >> 1] |= (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, at, 0, 0) << (16 * (e & 1));
                    else w[e] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
                }
                r[i] = u32x4{w[0], w[1], w[2], w[3]};
            }
            off += step;
        }
    }
    __device__ __forceinline__ void put(char* t, int tid) const {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int idx = tid + i * THREADS;
            *reinterpret_cast<u32x4*>(t + L::place(idx / L::kPieces, idx % L::kPieces)) = r[i];
        }
    }
    __device__ __forceinline__ void put_by_row(char* t, int tid) const {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int idx = tid + i * THREADS;
            L::put_by_row(t, idx / L::kPieces, idx % L::kPieces, r[i]);
        }
    }
    __device__ __forceinline__ bool bad() const {
        bool b = false;
#pragma unroll
        for (int i = 0; i < kMine; ++i) b |= piece_not_finite<T>(r[i]);
        return b;
    }
};

__device__ __forceinline__ Segment segment_of(const SegWord* segs, int64_t slot) {
    const int4 w = *reinterpret_cast<const int4*>(segs + slot);
    return Segment{w.x, w.y, w.z, w.w >> 2, (w.w & 1) != 0, (w.w & 2) != 0};
}
// kByBorder: the border that the segment begins at or, `behind`, ends at.
__device__ __forceinline__ int64_t state_base(const States& s, const Segment& seg, int len, bool behind, int head) {
    const int64_t unit = s.at == kByPage ? seg.page : s.at == kBySeq ? seg.seq : seg.row / len + (behind ? 1 : 0);
    return unit * s.unit + head * s.head;
}

// Workgroups go round the eight XCDs.  The value heads of a key head, which read
// the same q and k rows, follow one another on one XCD and share its L2; the
// slots, some of them empty, are spread over all XCDs evenly.
__device__ __forceinline__ int64_t xcd_item(int64_t b, int per) {
    const int64_t j = b >> 3;
    return ((j / per) * 8 + (b & 7)) * per + j % per;
}
inline int64_t xcd_grid(int64_t items, int per) { return (items / per + 7) / 8 * 8 * per; }

// What the decays of a chunk come to, in LDS.
struct Gates {
    float hi[64], lo[64];   // G, the inclusive sum of g in powers of two, as two floats
    float row[64];          // factor of an output row's state part
    float src[64];          // weight of a source row in the state's update
};

// Four values of an output row, the first at byte `at` of rs; VEC: all four
// exist, on whole vectors.
template <typename O, bool VEC> __device__ __forceinline__ void put4(__amdgpu_buffer_rsrc_t rs, uint32_t at, const f32x4& v, int nc) {
    if constexpr (VEC) {
        if constexpr (sizeof(O) == 4) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, at, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b64(u32x2{gdn::f32x2_to_bf16x2(v[0], v[1]), gdn::f32x2_to_bf16x2(v[2], v[3])}, rs, at, 0, 0);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t to = r < nc ? at + r * (uint32_t)sizeof(O) : kNowhere;
            if constexpr (sizeof(O) == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[r]), rs, to, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b16(gdn::f32_to_bf16(v[r]), rs, to, 0, 0);
        }
    }
}
// A wave's share of a chunk's output: 64 rows by 16 NT columns.
template <typename O, bool VEC, int NT>
__device__ __forceinline__ void put_rows(const AttendArgs& A, const f32x4 (&o)[4 * NT], int64_t row0, int head, int n, int col0, int g, int i) {
    const __amdgpu_buffer_rsrc_t rs = rows_buffer<O>(A.o, A.o_stride, row0, (int64_t)head * A.dv, n, A.dv);
    const uint32_t row = (uint32_t)A.o_stride * (uint32_t)sizeof(O);
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
        const int c4 = col0 + 16 * nn + 4 * g;
        const uint32_t at = (uint32_t)i * row + (uint32_t)c4 * (uint32_t)sizeof(O);
#pragma unroll
        for (int b = 0; b < 4; ++b) put4<O, VEC>(rs, c4 < A.dv ? at + 16 * b * row : kNowhere, o[b * NT + nn], A.dv - c4);
    }
}

// A chunk's bf16 rows from LDS, by the threads that later put the same pieces.
// QUADS: from where rows are put by row.
template <int W, int THREADS, bool VEC, bool QUADS>
__device__ __forceinline__ void flush_rows(const AttendArgs& A, const char* stage, int64_t row0, int head, int n, int tid) {
    using L = Tile<bf16_t, W>;
    constexpr int kMine = kChunk * L::kPieces / THREADS;
    const __amdgpu_buffer_rsrc_t rs = rows_buffer<bf16_t>(A.o, A.o_stride, row0, (int64_t)head * A.dv, n, A.dv);
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int idx = tid + k * THREADS, row = idx / L::kPieces, c = idx % L::kPieces * L::kElems;
        u32x4 v;
        if constexpr (QUADS) {
            const int to = L::quad(row, 2 * (idx % L::kPieces));
            const u32x2 lo = *reinterpret_cast<const u32x2*>(stage + to), hi = *reinterpret_cast<const u32x2*>(stage + (to ^ 16));
            v = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            v = *reinterpret_cast<const u32x4*>(stage + L::place(row, idx % L::kPieces));
        }
        const uint32_t at = ((uint32_t)row * (uint32_t)A.o_stride + (uint32_t)c) * 2u;
        if constexpr (VEC) {
            __builtin_amdgcn_raw_buffer_store_b128(v, rs, c < A.dv ? at : kNowhere, 0, 0);
        } else {
#pragma unroll
            for (int e = 0; e < L::kElems; ++e)
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v[e >> 1] >> (16 * (e & 1))), rs,
                                                      c + e < A.dv ? at + 2u * e : kNowhere, 0, 0);
        }
    }
}

template <typename T, int DK, int W, int NT, int MODE, bool BACK> struct Layout {
    static constexpr int DV = 16 * W * NT;
    static constexpr int kTerms = sizeof(T) == 2 ? 3 : 1;     // of P, S and the decayed v: all 24 bits
    static constexpr int kPTile = 64 * 4 * (int)sizeof(T);    // of one term
    static constexpr int kPTerm = kTri * kPTile;
    static constexpr bool kX = MODE == kDot || MODE == kDotRows;
    static constexpr bool kStage = sizeof(T) == 2 && MODE != kLocal;
    static constexpr int oK = 0;
    static constexpr int oV = oK + Tile<T, DK>::kBytes;
    static constexpr int oQ = oV + Tile<T, DV>::kBytes;
    static constexpr int oX = oQ + (MODE == kLocal ? 0 : Tile<T, DK>::kBytes);
    static constexpr int oFree = oX + (kX ? Tile<T, DV>::kBytes : 0);
    // With four bf16 tiles of 128 columns P takes the place of q, behind a barrier
    // of its own: two workgroups fit a compute unit only so.
    static constexpr bool kPOnQ = kX && sizeof(T) == 2 && DK == 128 && DV == 128;
    static constexpr int oP = kPOnQ ? oQ : oFree;
    static constexpr int oG = oFree + (MODE == kLocal || kPOnQ ? 0 : kTerms * kPTerm);
    // bf16 outputs leave through LDS as whole rows: where x's rows stood, or q's,
    // which the second half of a chunk does not need, else in a place of their own.
    static constexpr bool kStageOnQ = kStage && !kX && DK == DV;
    static constexpr int oOwn = oG + (int)sizeof(Gates);
    static constexpr int oO = kX ? oX : kStageOnQ ? oQ : oOwn;
    static constexpr int oBad = oOwn + (kStage && !kX && !kStageOnQ ? Tile<T, DV>::kBytes : 0);  // first row of a column that is not finite
    static constexpr bool kGuard = MODE == kAttend && !BACK;  // values that are not finite reach no row before theirs
    static constexpr int oDot = oBad + (kGuard ? DV * 8 + 16 : 0);
    static constexpr int oSum = oDot + (kX ? W * 64 * 4 : 0);
    static constexpr int kBytes = oSum + (MODE == kDotRows ? 64 * 4 * 4 : 0);
    static __device__ __forceinline__ char* stage_at(char* lds, int row, int c) {  // c a multiple of 4
        return lds + oO + (kStageOnQ ? Tile<T, DV>::quad(row, c / 4) : Tile<T, DV>::place(row, c / 8) + c % 8 * 2);
    }
    // Waves on a SIMD that the registers are cut for: what LDS has room for, four at
    // most; two for local sums of fp32 rows, which spill with four (16384 rows of 32
    // heads of 128 x 128: 189 us against 317).
    static constexpr int kRoom = 160 * 1024 / kBytes * W / 4;
    static constexpr int kMost = sizeof(T) == 4 && MODE == kLocal ? 2 : 4;
    static constexpr int kWavesPerSimd = kRoom < 1 ? 1 : kRoom > kMost ? kMost : kRoom;
};

// The state's rows 16 m + 4 g + r of one column, `at` from each other by rs;
// those that do not exist are zeros.
template <typename S, int M> __device__ __forceinline__ void load_state(f32x4 (&s)[M], const S* p, int rs, int dk, int g) {
    S raw[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) raw[m][r] = p[(int64_t)min(16 * m + 4 * g + r, dk - 1) * rs];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[m][r] = 16 * m + 4 * g + r < dk ? gdn::to_f32(raw[m][r]) : 0.0f;
}
template <typename S, int M> __device__ __forceinline__ void store_state(const f32x4 (&s)[M], S* p, int rs, int dk, int g, bool zero) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (16 * m + 4 * g + r < dk) p[(int64_t)(16 * m + 4 * g + r) * rs] = gdn::from_f32<S>(zero ? 0.0f : s[m][r]);
}

// W waves, 16 NT columns each.
template <typename T, int DK, int W, int NT, int MODE, bool back, bool VEC>
__global__ __launch_bounds__(64 * W, (Layout<T, DK, W, NT, MODE, back>::kWavesPerSimd)) void k_attend(const AttendArgs A) {
    using Y = Layout<T, DK, W, NT, MODE, back>;
    using TK = Tile<T, DK>;
    using TV = Tile<T, Y::DV>;
    // KG sums of the state's update in turn; fewer where a fourth tile's rows are in registers (with four kDotRows takes
    // 17 us more over 32768 rows of 32 heads, of 430)
    constexpr int KG = Y::kX ? 2 : 4, M = DK / 16, KS = DK / 32, TH = 64 * W;
    __shared__ __attribute__((aligned(16))) char lds[Y::kBytes];
    char* const tk = lds + Y::oK;
    char* const tv = lds + Y::oV;
    char* const tq = lds + Y::oQ;
    char* const tx = lds + Y::oX;
    char* const tp = lds + Y::oP;
    Gates& G = *reinterpret_cast<Gates*>(lds + Y::oG);
    int* const bad_row = reinterpret_cast<int*>(lds + Y::oBad);
    float* const poison = reinterpret_cast<float*>(bad_row + Y::DV);  // of a column's state, 0 or NaN
    int* const s_bad = bad_row + 2 * Y::DV;                       // some value of v is not finite
    float* const s_dot = reinterpret_cast<float*>(lds + Y::oDot);
    float* const s_sum = reinterpret_cast<float*>(lds + Y::oSum);

    const int64_t item = xcd_item(blockIdx.x, A.per);
    if (item >= A.n_slots * A.heads) return;
    const int64_t slot = item / A.heads;
    const int head = (int)(item - slot * A.heads);
    const Segment seg = segment_of(A.segs, slot);
    if (seg.rows <= 0) return;
    if (MODE == kLocal && (back ? seg.first : seg.last)) return;  // nothing follows

    const int lane0 = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col0 = wave * 16 * NT;
    const int n_chunks = (seg.rows + kChunk - 1) / kChunk;

    Fetch<T, DK, TH, VEC> fq, fk;
    Fetch<T, Y::DV, TH, VEC> fv, fx;
    float4 fg = make_float4(0, 0, 0, 0);
    float next_all = 0.0f;  // e^{G_C}
    auto fetch = [&](int c, int tid, int lane) {  // nothing where the segment has no chunk c
        const int64_t row0 = (int64_t)seg.row + (int64_t)c * kChunk;
        const int n = c < 0 ? 0 : min(kChunk, seg.rows - c * kChunk);
        fk.load(A.k, head, A.dk, row0, n, tid);
        fv.load(A.v, head, A.dv, row0, n, tid);
        if constexpr (MODE != kLocal) fq.load(A.q, head, A.dk, row0, n, tid);
        if constexpr (Y::kX) fx.load(A.x, head, A.dv, row0, n, tid);
        if (n > 0) {
            const float4* const rows = A.gates + (int64_t)head * A.n_rows + row0;
            if (wave == 0) fg = rows[min(lane, n - 1)];
            next_all = rows[n - 1].z;
        }
    };
    if constexpr (Y::kGuard) {
        if (threadIdx.x == 0) *s_bad = 0;
        for (int c = threadIdx.x; c < Y::DV; c += TH) poison[c] = 0.0f;
    }
    fetch(back ? n_chunks - 1 : 0, threadIdx.x, lane0);
    f32x4 S[NT][M];
    {
        const int g = lane0 >> 4, i = lane0 & 15;
        const States& in = !(back ? seg.last : seg.first)              ? A.mid
                           : !back && !seg.last && A.copy.at != kNoState ? A.copy
                                                                         : A.in;
        const bool zero = MODE == kLocal || in.at == kNoState ||
                          (in.at == kByPage && A.has_init && A.has_init[seg.seq] == 0);
        const int64_t base = zero ? 0 : state_base(in, seg, A.len, back, head);
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
            const int col = col0 + 16 * nn + i;
#pragma unroll
            for (int m = 0; m < M; ++m) S[nn][m] = f32x4{0, 0, 0, 0};
            if (!zero && col < A.dv) {
                const int64_t at = base + (int64_t)col * in.cs;
                if (in.bf16) load_state(S[nn], static_cast<const bf16_t*>(in.p) + at, in.rs, A.dk, g);
                else load_state(S[nn], static_cast<const float*>(in.p) + at, in.rs, A.dk, g);
            }
        }
    }
    lds_barrier();

    for (int step = 0; step < n_chunks; ++step) {
        const int c = back ? n_chunks - 1 - step : step;
        const int64_t row0 = (int64_t)seg.row + (int64_t)c * kChunk;
        const int n = min(kChunk, seg.rows - c * kChunk);
        // what follows from a lane's number is worked out again for each chunk: kept, it would fill the registers
        // (not so for the local sums: 110 us against 123 over 32768 rows of 32 heads)
        int lane = lane0;
        if constexpr (MODE != kLocal) asm volatile("" : "+v"(lane));
        const int tid = MODE == kLocal ? (int)threadIdx.x : wave * 64 + lane, g = lane >> 4, i = lane & 15;
        if constexpr (Y::kStage) {
            if (step > 0 && !A.o_f32)
                flush_rows<Y::DV, TH, VEC, Y::kStageOnQ>(A, lds + Y::oO, row0 + (back ? kChunk : -kChunk), head,
                                           back ? min(kChunk, seg.rows - (c + 1) * kChunk) : kChunk, tid);
        }
        const float all = next_all;
        fk.put(tk, tid);
        fv.put(tv, tid);
        if constexpr (MODE != kLocal) fq.put_by_row(tq, tid);
        if constexpr (Y::kX) fx.put(tx, tid);
        if (Y::kGuard && fv.bad()) *s_bad = 1;
        if (wave == 0) {  // rows behind the end count as the last one, whose weight is 1 and whose values are zeros
            G.hi[lane] = fg.x;
            G.lo[lane] = fg.y;
            G.row[lane] = A.f_i * (back ? fg.w : fg.z);
            G.src[lane] = A.f_u * (back ? fg.z : fg.w);
        }
        lds_barrier();
        // Where v is not finite (rare) zeros take its place, 0 times it being NaN:
        // outputs from its row on are overwritten, and the state's column is told.
        const bool bad = Y::kGuard && *s_bad != 0;
        if (bad) {
            for (int c2 = tid; c2 < Y::DV; c2 += TH) {
                int first = kChunk;
                for (int r = kChunk - 1; r >= 0; --r) {
                    T* const p = TV::at(tv, r, c2);
                    if (not_finite<T>(*p)) {
                        *p = 0;
                        first = r;
                    }
                }
                bad_row[c2] = first;
                poison[c2] = first < kChunk ? __uint_as_float(0x7fc00000u) : 0.0f;
            }
            lds_barrier();
        }

        f32x4 O[4 * NT];
        if constexpr (MODE != kLocal) {
            const int kr = TK::row_base(g, i), qr = TK::whole_base(g, i), xr = TV::row_base(g, i);
            // P: tile (y, x) of k q^T, decayed, in terms; the products of a wave's first tile are under way while
            // it multiplies q and S
            struct Of { int ty, tx; };
            auto tile_of = [](int t) {
                const int hi = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0, lo = t - hi * (hi + 1) / 2;
                return back ? Of{hi, lo} : Of{lo, hi};
            };
            auto products = [&](int t, f32x4 (&p)[2]) {
                const Of o = tile_of(t);
                p[0] = p[1] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) p[ks & 1] = mma(TK::by_row(tk, kr, o.ty, ks), TK::whole(tq, qr, o.tx, ks), p[ks & 1]);
            };
            auto decayed = [&](int t, f32x4 (&p)[2], float (&v)[4]) {
                const Of o = tile_of(t);
                settle(p);
                f32x4 pm[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
                if constexpr (MODE == kDotRows) {
#pragma unroll
                    for (int ks = 0; ks < Y::DV / 32; ++ks)
                        pm[ks & 1] = mma(TV::by_row(tv, xr, o.ty, ks), TV::by_row(tx, xr, o.tx, ks), pm[ks & 1]);
                }
                if constexpr (MODE == kDotRows) settle(pm);
                const int x = 16 * o.tx + i, y0 = 16 * o.ty + 4 * g;
                const float xh = G.hi[x], xl = G.lo[x];
                const f32x4 yh = *reinterpret_cast<const f32x4*>(G.hi + y0);
                const f32x4 yl = *reinterpret_cast<const f32x4*>(G.lo + y0);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float d = back ? (yh[r] - xh) + (yl[r] - xl) : (xh - yh[r]) + (xl - yl[r]);
                    const bool in = back ? y0 + r >= x : y0 + r <= x;
                    v[r] = in ? A.f_p * exp2_hw(d) * (p[0][r] + p[1][r]) : 0.0f;
                }
                if constexpr (MODE == kDotRows) {
                    // M without its diagonal: for a row x its sum over the tile's columns y, for a column y less its sum
                    // over the tile's rows x, at s_sum[row][the other tile]
                    float row = 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float m = y0 + r == x ? 0.0f : v[r] * (pm[0][r] + pm[1][r]);
                        row += m;
                        const float cs = reduce16(m);
                        if (i == 0) s_sum[(y0 + r) * 4 + o.tx] = -cs;
                    }
                    row += __shfl_xor(row, 16, 64);
                    row += __shfl_xor(row, 32, 64);
                    if (o.tx == o.ty) {  // written above by other lanes of this wave
                        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                        __builtin_amdgcn_wave_barrier();
                        row += s_sum[x * 4 + o.tx];
                    }
                    if (g == 0) s_sum[x * 4 + o.ty] = row;
                }
            };
            auto put = [&](int t, const float (&v)[4]) {
                const Of o = tile_of(t);
                const bool alone = is_alone<back>(o.tx, o.ty >> 1);
                char* const at = tp + pair<back>(o.tx, o.ty >> 1) * Y::kPTile + lane * ((alone ? 4 : 8) * (int)sizeof(T)) +
                                 (alone ? 0 : (o.ty & 1) * (4 * (int)sizeof(T)));
                if constexpr (sizeof(T) == 2) {
                    uint32_t a[3], b[3];
                    split2<3>(v[0], v[1], a);
                    split2<3>(v[2], v[3], b);
#pragma unroll
                    for (int j = 0; j < 3; ++j) *reinterpret_cast<u32x2*>(at + j * Y::kPTerm) = u32x2{a[j], b[j]};
                } else {
                    *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
                }
            };
            f32x4 p[2];
            if constexpr (MODE != kDotRows) products(wave, p);  // there, registers are short
            // the state's part, transposed: a lane holds four columns of row 16 b + i
#pragma unroll
            for (int j = 0; j < 4 * NT; ++j) O[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Frag<T> sf[NT][Y::kTerms], qf[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) qf[b] = TK::whole(tq, qr, b, ks);
#pragma unroll
                for (int nn = 0; nn < NT; ++nn) {
                    float f[8];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        f[r] = S[nn][2 * ks][r];
                        f[4 + r] = S[nn][2 * ks + 1][r];
                    }
                    split<Y::kTerms>(f, sf[nn]);
                }
#pragma unroll
                for (int ts = 0; ts < Y::kTerms; ++ts)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int nn = 0; nn < NT; ++nn) O[b * NT + nn] = mma(sf[nn][ts], qf[b], O[b * NT + nn]);
            }
            if constexpr (MODE == kDotRows) products(wave, p);
            float own[4];
            decayed(wave, p, own);
            // the tiles beyond W go to other waves, so to other SIMDs, in every chunk
            const int more = W + ((wave - 2 * step) & (W - 1));
            if constexpr (Y::kPOnQ) {
                static_assert(kTri <= 2 * W, "two tiles to a wave");
                float second[4];
                if (more < kTri) {
                    products(more, p);
                    decayed(more, p, second);
                }
                lds_barrier();  // q has been read
                put(wave, own);
                if (more < kTri) put(more, second);
            } else {
                put(wave, own);
                for (int t = more; t < kTri; t += W) {
                    products(t, p);
                    decayed(t, p, own);
                    put(t, own);
                }
            }
            settle(O);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float f = G.row[16 * b + i];
#pragma unroll
                for (int nn = 0; nn < NT; ++nn) O[b * NT + nn] *= f;
                if constexpr (Y::kX) {
                    float d = 0.0f;
#pragma unroll
                    for (int nn = 0; nn < NT; ++nn) {
                        const T* const p = TV::at(tx, 16 * b + i, col0 + 16 * nn + 4 * g);
#pragma unroll
                        for (int r = 0; r < 4; ++r) d = fmaf(O[b * NT + nn][r], gdn::to_f32(p[r]), d);
                    }
                    d += __shfl_xor(d, 16, 64);
                    d += __shfl_xor(d, 32, 64);
                    if (g == 0) s_dot[wave * 64 + 16 * b + i] = d;
                }
            }
            lds_barrier();  // P is whole
            if constexpr (Y::kX) {
                if (tid < n) {
                    float d = 0.0f;
#pragma unroll
                    for (int w = 0; w < W; ++w) d += s_dot[w * 64 + tid];
                    if constexpr (MODE == kDotRows) {
                        const f32x4 s = *reinterpret_cast<const f32x4*>(s_sum + 4 * tid);
                        d += (s[0] + s[1]) + (s[2] + s[3]);
                    }
                    A.dot[(int64_t)head * A.n_rows + row0 + tid] = d;
                }
            }
        }
        const int vc = TV::col_base(g, i);
        if constexpr (MODE != kLocal) {  // P v, and the chunk's output is whole
#pragma unroll
            for (int ys = 0; ys < 2; ++ys) {
                Frag<T> vf[NT];
#pragma unroll
                for (int nn = 0; nn < NT; ++nn) vf[nn] = TV::by_col(tv, vc, ys, wave * NT + nn);
#pragma unroll
                for (int j = 0; j < Y::kTerms; ++j)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (!is_pair<back>(b, ys)) continue;
                        const bool alone = is_alone<back>(b, ys);
                        const char* const p = tp + j * Y::kPTerm + pair<back>(b, ys) * Y::kPTile + lane * ((alone ? 4 : 8) * (int)sizeof(T));
                        Frag<T> pf;
                        if constexpr (sizeof(T) == 2) {
                            if (alone) {
                                const u32x2 a = *reinterpret_cast<const u32x2*>(p);
                                pf.v = back ? u32x4{0, 0, a.x, a.y} : u32x4{a.x, a.y, 0, 0};
                            } else {
                                pf.v = *reinterpret_cast<const u32x4*>(p);
                            }
                        } else {
                            const f32x4 none = {0, 0, 0, 0}, one = *reinterpret_cast<const f32x4*>(p);
                            const f32x4 a = alone && back ? none : one;
                            const f32x4 c2 = alone ? (back ? one : none) : *reinterpret_cast<const f32x4*>(p + 16);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                pf.v[e] = a[e];
                                pf.v[4 + e] = c2[e];
                            }
                        }
#pragma unroll
                        for (int nn = 0; nn < NT; ++nn) O[b * NT + nn] = mma(vf[nn], pf, O[b * NT + nn]);
                    }
            }
            settle(O);
            if (!Y::kStage || A.o_f32) {
                put_rows<float, VEC, NT>(A, O, row0, head, n, col0, g, i);
            } else {
#pragma unroll
                for (int nn = 0; nn < NT; ++nn)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        *reinterpret_cast<u32x2*>(Y::stage_at(lds, 16 * b + i, col0 + 16 * nn + 4 * g)) =
                            u32x2{gdn::f32x2_to_bf16x2(O[b * NT + nn][0], O[b * NT + nn][1]),
                                  gdn::f32x2_to_bf16x2(O[b * NT + nn][2], O[b * NT + nn][3])};
            }
            if (bad) {  // the same lanes wrote these places before
                const bool staged = Y::kStage && !A.o_f32;
                const __amdgpu_buffer_rsrc_t rs = rows_buffer<float>(A.o, A.o_stride, row0, (int64_t)head * A.dv, staged ? 0 : n, A.dv);
                for (int nn = 0; nn < NT; ++nn)
                    for (int r = 0; r < 4; ++r) {
                        const int c2 = col0 + 16 * nn + 4 * g + r;
                        for (int x = i; x < kChunk; x += 16) {
                            if (x < bad_row[c2]) continue;
                            if (staged) {
                                reinterpret_cast<bf16_t*>(Y::stage_at(lds, x, c2 - r))[r] = 0x7fc0;
                            } else {
                                const uint32_t at = ((uint32_t)x * (uint32_t)A.o_stride + (uint32_t)c2) * (uint32_t)sizeof(float);
                                __builtin_amdgcn_raw_buffer_store_b32(0x7fc00000u, rs, c2 < A.dv ? at : kNowhere, 0, 0);
                            }
                        }
                    }
            }
        }
        // The next chunk's rows are asked for where the registers that held the output are free.
        fetch(back ? c - 1 : c + 1, tid, lane);
        const int kc = TK::col_base(g, i);
        auto weighed = [&](int ys, Frag<T> (&vw)[NT][Y::kTerms]) {  // v's rows with their decays
            const f32x4 w0 = *reinterpret_cast<const f32x4*>(G.src + 32 * ys + 4 * g);
            const f32x4 w1 = *reinterpret_cast<const f32x4*>(G.src + 32 * ys + 16 + 4 * g);
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) {
                float f[8];
                values(TV::by_col(tv, vc, ys, wave * NT + nn), f);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    f[r] *= w0[r];
                    f[4 + r] *= w1[r];
                }
                if constexpr (Y::kGuard) f[0] += poison[col0 + 16 * nn + i];
                split<Y::kTerms>(f, vw[nn]);
            }
        };
        if constexpr (sizeof(T) == 4) {
            // The chunk's sum by itself, then one rounding at the state's size: over
            // 1500 rows a state's error 1.9e-7 -> 1.2e-7 of it, for 1% of the time with
            // states of 128 x 128 and 3% with 64 x 64; four chains reach 1.0e-7 for 8%.
            Frag<T> vw[2][NT][1];
            weighed(0, vw[0]);
            weighed(1, vw[1]);
#pragma unroll
            for (int m = 0; m < M; m += 2) {
                f32x4 sum[2 * NT * 2] = {};
#pragma unroll
                for (int ys = 0; ys < 2; ++ys)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const Frag<T> kf = TK::by_col(tk, kc, ys, m + j);
#pragma unroll
                        for (int nn = 0; nn < NT; ++nn)
                            mma_chains(kf, vw[ys][nn][0], *reinterpret_cast<f32x4(*)[2]>(sum + 2 * (2 * nn + j)));
                    }
                settle(sum);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nn = 0; nn < NT; ++nn) {
                        const f32x4 own = sum[2 * (2 * nn + j)] + sum[2 * (2 * nn + j) + 1];
#pragma unroll
                        for (int r = 0; r < 4; ++r) S[nn][m + j][r] = fmaf(S[nn][m + j][r], all, own[r]);
                    }
            }
        } else {
#pragma unroll
            for (int nn = 0; nn < NT; ++nn)
#pragma unroll
                for (int m = 0; m < M; ++m) S[nn][m] *= all;
#pragma unroll
            for (int ys = 0; ys < 2; ++ys) {
                Frag<T> vw[NT][Y::kTerms];
                weighed(ys, vw);
#pragma unroll
                for (int m = 0; m < M; m += KG) {  // sums in turn: none waits for itself
                    Frag<T> kf[KG];
#pragma unroll
                    for (int j = 0; j < KG; ++j) kf[j] = TK::by_col(tk, kc, ys, m + j);
#pragma unroll
                    for (int tt = 0; tt < Y::kTerms; ++tt)
#pragma unroll
                        for (int j = 0; j < KG; ++j)
#pragma unroll
                            for (int nn = 0; nn < NT; ++nn) S[nn][m + j] = mma(kf[j], vw[nn][tt], S[nn][m + j]);
                }
            }
        }
        if (bad) {
            lds_barrier();
            if (tid == 0) *s_bad = 0;
            for (int c2 = tid; c2 < Y::DV; c2 += TH) poison[c2] = 0.0f;
        }
        lds_barrier();  // the tiles are free
    }

    if constexpr (Y::kStage) {
        const int c = back ? 0 : n_chunks - 1;
        if (!A.o_f32)
            flush_rows<Y::DV, TH, VEC, Y::kStageOnQ>(A, lds + Y::oO, (int64_t)seg.row + (int64_t)c * kChunk, head,
                                       min(kChunk, seg.rows - c * kChunk), threadIdx.x);
    }
    if (A.out.at != kNoState && (MODE == kLocal || (back ? seg.first : seg.last))) {
        const bool zero = A.zero_uninit && A.has_init && A.has_init[seg.seq] == 0;
        const int64_t base = state_base(A.out, seg, A.len, !back, head);
        const int g = lane0 >> 4, i = lane0 & 15;
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
            const int col = col0 + 16 * nn + i;
            settle(S[nn]);
            if (col < A.dv) {
                const int64_t at = base + (int64_t)col * A.out.cs;
                if (A.out.bf16) store_state(S[nn], static_cast<bf16_t*>(A.out.p) + at, A.out.rs, A.dk, g, zero);
                else store_state(S[nn], static_cast<float*>(A.out.p) + at, A.out.rs, A.dk, g, zero);
            }
        }
    }
}

template <typename T, int DK, int W, int NT, int MODE, bool BACK, bool VEC> hipError_t run_attend(const AttendArgs& a, hipStream_t s) {
    static_assert(Layout<T, DK, W, NT, MODE, BACK>::kBytes <= 160 * 1024, "LDS");
    const int64_t grid = xcd_grid(a.n_slots * a.heads, a.per);
    hipLaunchKernelGGL((k_attend<T, DK, W, NT, MODE, BACK, VEC>), dim3((unsigned)grid), dim3(64 * W), 0, s, a);
    return hipGetLastError();
}
template <typename T, int MODE, bool BACK, bool VEC> hipError_t pick_attend(const AttendArgs& a, hipStream_t s) {
    constexpr int W = 8, NT = 1;  // for 128 columns
    if (a.dk <= 64)
        return a.dv <= 64 ? run_attend<T, 64, 4, 1, MODE, BACK, VEC>(a, s) : run_attend<T, 64, W, NT, MODE, BACK, VEC>(a, s);
    return a.dv <= 64 ? run_attend<T, 128, 4, 1, MODE, BACK, VEC>(a, s) : run_attend<T, 128, W, NT, MODE, BACK, VEC>(a, s);
}
template <typename T, int MODE, bool BACK> hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
    return a.vec ? pick_attend<T, MODE, BACK, true>(a, s) : pick_attend<T, MODE, BACK, false>(a, s);
}

}  // namespace gdnl
