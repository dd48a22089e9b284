// gdnl_attend.hpp -- linear attention over chunks of 64 rows on matrix cores,
// forward or backward in time (AttendArgs), for one act type.
//
// A workgroup of four waves walks a segment's chunks for one value head; a
// wave owns 16 NT columns of the head's state S, all DK rows of them, in the
// accumulators, so S never leaves the registers.  Matrix products reduce over
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
// Decays.  G is summed within a chunk in 64 bits and kept as two floats, so
// e^{G_x - G_y} is good to the difference's own digits; it is set, not
// multiplied, to zero where y lies ahead of x.  g ends at -128, where e^g is 0:
// differences of the rows behind it stay finite.
//
// Roundings with bf16 rows.  The products of q, k and v themselves are exact.
// What is not a bf16 number is split into terms of eight bits: P into two (2^-16
// of its value is left, far below the output's 2^-9), S into two for o and three
// where the gates' gradient needs fp32, and the decayed rows of the state's
// update into three (nothing is left): a state is as good as its fp32 sum.
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

constexpr int kWaves = kThreads / 64;
constexpr int kTri = 10;  // tiles of 16 x 16 on or below the diagonal of 64 x 64

__device__ __forceinline__ int tri(int lo, int hi) { return hi * (hi + 1) / 2 + lo; }

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
// row is exclusive-ored by the row: both readings below spread over all banks.
template <typename T, int W> struct Tile {
    static constexpr int kPieces = W * (int)sizeof(T) / 16;           // of a row
    static constexpr int kMine = kChunk * kPieces / kThreads;        // of a thread
    static constexpr int kElems = 16 / (int)sizeof(T);
    static constexpr int kBytes = kChunk * W * (int)sizeof(T);
    static __device__ __forceinline__ int place(int row, int piece) {
        const int x = sizeof(T) == 4 ? (row & 15) : W == 128 ? (row & 7) << 1 : ((row >> 1) & 3) << 1;
        return row * (W * (int)sizeof(T)) + ((piece ^ x) << 4);
    }
    // positions 4g..4g+3 of the 16s at 32 ks and 32 ks + 16, of row `row`
    static __device__ __forceinline__ Frag<T> row_frag(const char* t, int row, int ks, int g) {
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            const u32x2 a = *reinterpret_cast<const u32x2*>(t + place(row, 4 * ks + (g >> 1)) + (g & 1) * 8);
            const u32x2 b = *reinterpret_cast<const u32x2*>(t + place(row, 4 * ks + 2 + (g >> 1)) + (g & 1) * 8);
            f.v = u32x4{a.x, a.y, b.x, b.y};
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4*>(t + place(row, 8 * ks + g));
            const f32x4 b = *reinterpret_cast<const f32x4*>(t + place(row, 8 * ks + 4 + g));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f.v[e] = a[e];
                f.v[4 + e] = b[e];
            }
        }
        return f;
    }
    // rows 4g..4g+3 of the 16s at 32 ys and 32 ys + 16, of column c0 + i
    static __device__ __forceinline__ Frag<T> col_frag(const char* t, int ys, int c0, int g, int i) {
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            // lanes 4j..4j+3 of a group of 16 name row 4g + j, 16 columns of it; each lane receives a column
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const int row = 32 * ys + 4 * g + (i >> 2), piece = (c0 >> 3) + ((i & 3) >> 1), in = (i & 1) * 8;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + place(row, piece) + in));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + place(row + 16, piece) + in));
            const u32x2 a2 = __builtin_bit_cast(u32x2, a), b2 = __builtin_bit_cast(u32x2, b);
            f.v = u32x4{a2.x, a2.y, b2.x, b2.y};
        } else {
            const int c = c0 + i;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 32 * ys + 16 * (e >> 2) + 4 * g + (e & 3);
                f.v[e] = *reinterpret_cast<const float*>(t + place(row, c >> 2) + (c & 3) * 4);
            }
        }
        return f;
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
template <typename T> __device__ __forceinline__ bool piece_not_finite(uint4 p) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) any |= ((w[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        else any |= ((w[i] & 0x7f800000u) + 0x00800000u) & 0x80000000u;
    }
    return any != 0;
}

// A thread's pieces of 64 rows of a head, on their way to LDS.  Rows from n on
// and columns from d on are zeros.
template <typename T, int W> struct Fetch {
    using L = Tile<T, W>;
    uint4 r[L::kMine];
    __device__ __forceinline__ void load(const Rows& R, int head, int d, int64_t row0, int n, int tid) {
        const T* base = static_cast<const T*>(R.p) + row0 * R.stride + (int64_t)(head / R.per) * d;
#pragma unroll
        for (int i = 0; i < L::kMine; ++i) {
            const int idx = tid + i * kThreads, row = idx / L::kPieces, c = idx % L::kPieces * L::kElems;
            r[i] = make_uint4(0, 0, 0, 0);
            if (row < n && c < d) {
                const T* p = base + row * R.stride + c;
                if (R.vec) {
                    r[i] = *reinterpret_cast<const uint4*>(p);
                } else {
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < L::kElems; ++e) {
                        if (c + e < d) {
                            if constexpr (sizeof(T) == 2) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
                            else w[e] = __float_as_uint(p[e]);
                        }
                    }
                    r[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    }
    __device__ __forceinline__ void put(char* t, int tid) const {
#pragma unroll
        for (int i = 0; i < L::kMine; ++i) {
            const int idx = tid + i * kThreads;
            *reinterpret_cast<uint4*>(t + L::place(idx / L::kPieces, idx % L::kPieces)) = r[i];
        }
    }
    __device__ __forceinline__ bool bad() const {
        bool b = false;
#pragma unroll
        for (int i = 0; i < L::kMine; ++i) b |= piece_not_finite<T>(r[i]);
        return b;
    }
};

__device__ __forceinline__ Segment segment_of(const SegWord* segs, int64_t slot) {
    const int4 w = *reinterpret_cast<const int4*>(segs + slot);
    return Segment{w.x, w.y, w.z, w.w >> 2, (w.w & 1) != 0, (w.w & 2) != 0};
}
__device__ __forceinline__ int64_t state_base(const States& s, const Segment& seg, int64_t slot, int head) {
    const int64_t unit = s.at == kByPage ? seg.page : s.at == kBySeq ? seg.seq : slot;
    return unit * s.unit + head * s.head;
}

// Workgroups go round the eight XCDs; each XCD takes a run of consecutive
// (slot, head) pairs, so the value heads that read the same q and k rows, and
// a segment's neighbours, share an L2.
__device__ __forceinline__ int64_t xcd_item(int64_t b, int64_t n) {
    const int64_t per = (n + 7) / 8;
    return (b & 7) * per + (b >> 3);
}
inline int64_t xcd_grid(int64_t n) { return (n + 7) / 8 * 8; }

template <typename T, int DK, int NT, int MODE> struct Layout {
    static constexpr int DV = 64 * NT;
    static constexpr int kTermsP = sizeof(T) == 2 ? 2 : 1;
    static constexpr int kTermsV = sizeof(T) == 2 ? 3 : 1;
    static constexpr int kTermsS = sizeof(T) == 4 ? 1 : MODE == kAttend ? 2 : 3;
    static constexpr int kPTile = 64 * 4 * (int)sizeof(T);
    static constexpr bool kX = MODE == kDot || MODE == kDotRows;
    static constexpr int oK = 0;
    static constexpr int oV = oK + Tile<T, DK>::kBytes;
    static constexpr int oQ = oV + Tile<T, DV>::kBytes;
    static constexpr int oX = oQ + (MODE == kLocal ? 0 : Tile<T, DK>::kBytes);
    static constexpr int oP = oX + (kX ? Tile<T, DV>::kBytes : 0);
    static constexpr int oG = oP + (MODE == kLocal ? 0 : kTri * kTermsP * kPTile);  // G (two floats), row factors, weights, e^{G_C}
    static constexpr int oBad = oG + 4 * 64 * 4 + 16;                               // first row of a column that is not finite
    static constexpr int oDot = oBad + DV * 4;
    static constexpr int oSum = oDot + (kX ? kWaves * 64 * 4 : 0);
    static constexpr int kBytes = oSum + (MODE == kDotRows ? kTri * 32 * 4 : 0);
};

template <typename T, int DK, int NT, int MODE>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void k_attend(const AttendArgs A) {
    using Y = Layout<T, DK, NT, MODE>;
    using TK = Tile<T, DK>;
    using TV = Tile<T, Y::DV>;
    constexpr int M = DK / 16, KS = DK / 32;
    __shared__ __attribute__((aligned(16))) char lds[Y::kBytes];
    char* const tk = lds + Y::oK;
    char* const tv = lds + Y::oV;
    char* const tq = lds + Y::oQ;
    char* const tx = lds + Y::oX;
    char* const tp = lds + Y::oP;
    float* const g_hi = reinterpret_cast<float*>(lds + Y::oG);
    float* const g_lo = g_hi + 64;
    float* const g_row = g_hi + 128;   // factor of an output row's state part
    float* const g_src = g_hi + 192;   // weight of a source row in the update
    float* const g_all = g_hi + 256;   // e^{G_C}; then: some value of v is not finite
    int* const s_bad = reinterpret_cast<int*>(g_hi + 257);
    int* const bad_row = reinterpret_cast<int*>(lds + Y::oBad);
    float* const s_dot = reinterpret_cast<float*>(lds + Y::oDot);
    float* const s_sum = reinterpret_cast<float*>(lds + Y::oSum);

    const int64_t item = xcd_item(blockIdx.x, A.n_slots * A.heads);
    if (item >= A.n_slots * A.heads) return;
    const int64_t slot = item / A.heads;
    const int head = (int)(item - slot * A.heads);
    const Segment seg = segment_of(A.segs, slot);
    if (seg.rows <= 0) return;
    if (MODE == kLocal && (A.back ? seg.first : seg.last)) return;  // nothing follows

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, i = lane & 15;
    const int col0 = wave * 16 * NT;
    const bool back = A.back != 0;

    f32x4 S[M][NT];
    {
        const bool zero = MODE == kLocal || A.in.at == kNoState ||
                          (A.in.at == kByPage && A.has_init && A.has_init[seg.seq] == 0);
        const int64_t base = zero ? 0 : state_base(A.in, seg, slot, head);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * m + 4 * g + r, col = col0 + 16 * n + i;
                    float v = 0.0f;
                    if (!zero && row < A.dk && col < A.dv) {
                        const int64_t at = base + (int64_t)row * A.in.rs + (int64_t)col * A.in.cs;
                        v = A.in.bf16 ? gdn::to_f32(static_cast<const bf16_t*>(A.in.p)[at])
                                      : static_cast<const float*>(A.in.p)[at];
                    }
                    S[m][n][r] = v;
                }
    }

    const int n_chunks = (seg.rows + kChunk - 1) / kChunk;
    Fetch<T, DK> fq, fk;
    Fetch<T, Y::DV> fv, fx;
    float fg = 0.0f;
    auto fetch = [&](int c) {
        const int64_t row0 = (int64_t)seg.row + (int64_t)c * kChunk;
        const int n = min(kChunk, seg.rows - c * kChunk);
        fk.load(A.k, head, A.dk, row0, n, tid);
        fv.load(A.v, head, A.dv, row0, n, tid);
        if constexpr (MODE != kLocal) fq.load(A.q, head, A.dk, row0, n, tid);
        if constexpr (Y::kX) fx.load(A.x, head, A.dv, row0, n, tid);
        fg = lane < n ? A.g[(row0 + lane) * A.g_stride + head] : 0.0f;
    };
    if (tid == 0) *s_bad = 0;
    for (int c = tid; c < Y::DV; c += kThreads) bad_row[c] = kChunk;
    fetch(back ? n_chunks - 1 : 0);
    double total = 0.0;
    lds_barrier();

    for (int step = 0; step < n_chunks; ++step) {
        const int c = back ? n_chunks - 1 - step : step;
        const int64_t row0 = (int64_t)seg.row + (int64_t)c * kChunk;
        const int n = min(kChunk, seg.rows - c * kChunk);
        fk.put(tk, tid);
        fv.put(tv, tid);
        if constexpr (MODE != kLocal) fq.put(tq, tid);
        if constexpr (Y::kX) fx.put(tx, tid);
        if (fv.bad()) *s_bad = 1;
        if (wave == 0) {
            const float gv = fg < -128.0f ? -128.0f : fg;  // a NaN stays
            double G = (double)gv * 1.4426950408889634;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double up = __shfl_up(G, d, 64);
                if (lane >= d) G += up;
            }
            const double GC = __shfl(G, 63, 64);
            total += GC;
            const float hi = (float)G, lo = (float)(G - (double)hi);
            const float into = (float)G, rest = (float)(GC - G);
            const float e_into = exp2_hw(into) * (1.0f + 0.6931472f * (float)(G - (double)into));
            const float e_rest = exp2_hw(rest) * (1.0f + 0.6931472f * (float)((GC - G) - (double)rest));
            g_hi[lane] = hi;
            g_lo[lane] = lo;
            g_row[lane] = A.f_i * (back ? e_rest : e_into);
            g_src[lane] = A.f_u * (back ? e_into : e_rest);
            if (lane == 63) *g_all = e_into;
        }
        lds_barrier();
        const bool bad = !back && *s_bad != 0;  // rare
        if (bad) {
            for (int c2 = tid; c2 < Y::DV; c2 += kThreads) {
                int first = kChunk;
                for (int r = 0; r < kChunk; ++r) {
                    T* p = TV::at(tv, r, c2);
                    if (not_finite<T>(*p)) {
                        *p = 0;
                        first = min(first, r);
                    }
                }
                bad_row[c2] = first;
            }
            lds_barrier();
        }
        if (step + 1 < n_chunks) fetch(back ? c - 1 : c + 1);

        f32x4 O[4 * NT];
        if constexpr (MODE != kLocal) {
            // P: tile (y, x) of k q^T, decayed, as two terms
            for (int t = wave; t < kTri; t += kWaves) {
                const int hi = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0, lo = t - hi * (hi + 1) / 2;
                const int ty = back ? hi : lo, tx_ = back ? lo : hi;
                if (16 * hi >= n) continue;
                f32x4 p[1] = {f32x4{0, 0, 0, 0}};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    p[0] = mma(TK::row_frag(tk, 16 * ty + i, ks, g), TK::row_frag(tq, 16 * tx_ + i, ks, g), p[0]);
                f32x4 pm[1] = {f32x4{0, 0, 0, 0}};
                if constexpr (MODE == kDotRows) {
#pragma unroll
                    for (int ks = 0; ks < Y::DV / 32; ++ks)
                        pm[0] = mma(TV::row_frag(tv, 16 * ty + i, ks, g), TV::row_frag(tx, 16 * tx_ + i, ks, g), pm[0]);
                    settle(pm);
                }
                settle(p);
                const int x = 16 * tx_ + i, y0 = 16 * ty + 4 * g;
                const float xh = g_hi[x], xl = g_lo[x];
                const f32x4 yh = *reinterpret_cast<const f32x4*>(g_hi + y0);
                const f32x4 yl = *reinterpret_cast<const f32x4*>(g_lo + y0);
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float d = back ? (yh[r] - xh) + (yl[r] - xl) : (xh - yh[r]) + (xl - yl[r]);
                    const bool in = back ? y0 + r >= x : y0 + r <= x;
                    v[r] = in ? A.f_p * exp2_hw(d) * p[0][r] : 0.0f;
                }
                char* const at = tp + t * (Y::kTermsP * Y::kPTile) + lane * (4 * (int)sizeof(T));
                if constexpr (sizeof(T) == 2) {
                    uint32_t a[2], b[2];
                    split2<2>(v[0], v[1], a);
                    split2<2>(v[2], v[3], b);
#pragma unroll
                    for (int j = 0; j < 2; ++j) *reinterpret_cast<u32x2*>(at + j * Y::kPTile) = u32x2{a[j], b[j]};
                } else {
                    *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
                }
                if constexpr (MODE == kDotRows) {
                    // M without its diagonal: sums over the tile's columns y for a row x, over its rows x for a column y
                    float row = 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float m = y0 + r == x ? 0.0f : v[r] * pm[0][r];
                        row += m;
                        const float col = reduce16(m);
                        if (i == 0) s_sum[t * 32 + 16 + 4 * g + r] = col;
                    }
                    row += __shfl_xor(row, 16, 64);
                    row += __shfl_xor(row, 32, 64);
                    if (g == 0) s_sum[t * 32 + i] = row;
                }
            }
            // the state's part
#pragma unroll
            for (int j = 0; j < 4 * NT; ++j) O[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Frag<T> sf[NT][Y::kTermsS];
#pragma unroll
                for (int nn = 0; nn < NT; ++nn) {
                    float f[8];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        f[r] = S[2 * ks][nn][r];
                        f[4 + r] = S[2 * ks + 1][nn][r];
                    }
                    split<Y::kTermsS>(f, sf[nn]);
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const Frag<T> qf = TK::row_frag(tq, 16 * b + i, ks, g);
#pragma unroll
                    for (int nn = 0; nn < NT; ++nn)
#pragma unroll
                        for (int ts = 0; ts < Y::kTermsS; ++ts) O[b * NT + nn] = mma(qf, sf[nn][ts], O[b * NT + nn]);
                }
            }
            settle(O);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const f32x4 f = *reinterpret_cast<const f32x4*>(g_row + 16 * b + 4 * g);
#pragma unroll
                for (int nn = 0; nn < NT; ++nn) O[b * NT + nn] *= f;
                if constexpr (Y::kX) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float d = 0.0f;
#pragma unroll
                        for (int nn = 0; nn < NT; ++nn)
                            d = fmaf(O[b * NT + nn][r], gdn::to_f32(*TV::at(tx, 16 * b + 4 * g + r, col0 + 16 * nn + i)), d);
                        d = reduce16(d);
                        if (i == 0) s_dot[wave * 64 + 16 * b + 4 * g + r] = d;
                    }
                }
            }
            lds_barrier();  // P is whole
            if constexpr (Y::kX) {
                if (tid < n) {
                    float d = (s_dot[tid] + s_dot[64 + tid]) + (s_dot[128 + tid] + s_dot[192 + tid]);
                    if constexpr (MODE == kDotRows) {
                        const int b = tid >> 4, k = tid & 15;
                        float row = 0.0f, col = 0.0f;
                        for (int o = 0; o < 4; ++o) {  // the other tile's index
                            if (16 * max(o, b) >= n) break;
                            if (back ? o >= b : o <= b) row += s_sum[tri(min(o, b), max(o, b)) * 32 + k];
                            if (back ? o <= b : o >= b) col += s_sum[tri(min(o, b), max(o, b)) * 32 + 16 + k];
                        }
                        d += row - col;
                    }
                    A.dot[(int64_t)head * A.n_rows + row0 + tid] = d;
                }
            }
        }

        // P v, and the state's update from the same v
        const float all = *g_all;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) S[m][nn] *= all;
#pragma unroll
        for (int ys = 0; ys < 2; ++ys) {
            if (32 * ys >= n) break;
            Frag<T> vf[NT], vw[NT][Y::kTermsV];
            const f32x4 w0 = *reinterpret_cast<const f32x4*>(g_src + 32 * ys + 4 * g);
            const f32x4 w1 = *reinterpret_cast<const f32x4*>(g_src + 32 * ys + 16 + 4 * g);
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) {
                vf[nn] = TV::col_frag(tv, ys, col0 + 16 * nn, g, i);
                float f[8];
                values(vf[nn], f);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    f[r] *= w0[r];
                    f[4 + r] *= w1[r];
                }
                split<Y::kTermsV>(f, vw[nn]);
            }
            if constexpr (MODE != kLocal) {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const bool lower = back ? 2 * ys >= b : 2 * ys <= b, upper = back ? 2 * ys + 1 >= b : 2 * ys + 1 <= b;
                    const bool is_lower = lower && 16 * max(2 * ys, b) < n, is_upper = upper && 16 * max(2 * ys + 1, b) < n;
                    if (!is_lower && !is_upper) continue;
                    const int t0 = tri(min(2 * ys, b), max(2 * ys, b)), t1 = tri(min(2 * ys + 1, b), max(2 * ys + 1, b));
#pragma unroll
                    for (int j = 0; j < Y::kTermsP; ++j) {
                        Frag<T> pf;
                        const char* const p0 = tp + (t0 * Y::kTermsP + j) * Y::kPTile + lane * (4 * (int)sizeof(T));
                        const char* const p1 = tp + (t1 * Y::kTermsP + j) * Y::kPTile + lane * (4 * (int)sizeof(T));
                        if constexpr (sizeof(T) == 2) {
                            const u32x2 a = is_lower ? *reinterpret_cast<const u32x2*>(p0) : u32x2{0, 0};
                            const u32x2 bb = is_upper ? *reinterpret_cast<const u32x2*>(p1) : u32x2{0, 0};
                            pf.v = u32x4{a.x, a.y, bb.x, bb.y};
                        } else {
                            const f32x4 z = {0, 0, 0, 0};
                            const f32x4 a = is_lower ? *reinterpret_cast<const f32x4*>(p0) : z;
                            const f32x4 bb = is_upper ? *reinterpret_cast<const f32x4*>(p1) : z;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                pf.v[e] = a[e];
                                pf.v[4 + e] = bb[e];
                            }
                        }
#pragma unroll
                        for (int nn = 0; nn < NT; ++nn) O[b * NT + nn] = mma(pf, vf[nn], O[b * NT + nn]);
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const Frag<T> kf = TK::col_frag(tk, ys, 16 * m, g, i);
#pragma unroll
                for (int nn = 0; nn < NT; ++nn)
#pragma unroll
                    for (int tt = 0; tt < Y::kTermsV; ++tt) S[m][nn] = mma(kf, vw[nn][tt], S[m][nn]);
            }
        }
        if constexpr (MODE != kLocal) {
            settle(O);
            if (bad) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int nn = 0; nn < NT; ++nn) {
                        const int first = bad_row[col0 + 16 * nn + i];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int x = 16 * b + 4 * g + r;
                            if (x >= first) O[b * NT + nn][r] = __uint_as_float(0x7fc00000u);
                        }
                    }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int nn = 0; nn < NT; ++nn) {
                    const int col = col0 + 16 * nn + i;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int x = 16 * b + 4 * g + r;
                        if (x < n && col < A.dv) {
                            const int64_t at = (row0 + x) * A.o_stride + (int64_t)head * A.dv + col;
                            if (A.o_f32) static_cast<float*>(A.o)[at] = O[b * NT + nn][r];
                            else static_cast<T*>(A.o)[at] = gdn::from_f32<T>(O[b * NT + nn][r]);
                        }
                    }
                }
        }
        if (bad) {  // the column is not a number from here on
#pragma unroll
            for (int nn = 0; nn < NT; ++nn)
                if (bad_row[col0 + 16 * nn + i] != kChunk) {
#pragma unroll
                    for (int m = 0; m < M; ++m)
#pragma unroll
                        for (int r = 0; r < 4; ++r) S[m][nn][r] = __uint_as_float(0x7fc00000u);
                }
            lds_barrier();
            if (tid == 0) *s_bad = 0;
            for (int c2 = tid; c2 < Y::DV; c2 += kThreads) bad_row[c2] = kChunk;
        }
        lds_barrier();  // the tiles are free
    }

    const bool write = A.out.at != kNoState && (MODE == kLocal || (back ? seg.first : seg.last));
    if (write) {
#pragma unroll
        for (int m = 0; m < M; ++m) settle(S[m]);
        const bool zero = A.zero_uninit && A.has_init && A.has_init[seg.seq] == 0;
        const int64_t base = state_base(A.out, seg, slot, head);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int nn = 0; nn < NT; ++nn)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * m + 4 * g + r, col = col0 + 16 * nn + i;
                    if (row < A.dk && col < A.dv) {
                        const int64_t at = base + (int64_t)row * A.out.rs + (int64_t)col * A.out.cs;
                        const float v = zero ? 0.0f : S[m][nn][r];
                        if (A.out.bf16) static_cast<bf16_t*>(A.out.p)[at] = gdn::f32_to_bf16(v);
                        else static_cast<float*>(A.out.p)[at] = v;
                    }
                }
    }
    if (MODE == kLocal && tid == 0) A.total[slot * A.heads + head] = total;
}

template <typename T, int DK, int NT, int MODE> hipError_t run_attend(const AttendArgs& a, hipStream_t s) {
    static_assert(Layout<T, DK, NT, MODE>::kBytes <= 160 * 1024, "LDS");
    const int64_t grid = xcd_grid(a.n_slots * a.heads);
    hipLaunchKernelGGL((k_attend<T, DK, NT, MODE>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
template <typename T, int MODE> hipError_t pick_attend(const AttendArgs& a, hipStream_t s) {
    if (a.dk <= 64) return a.dv <= 64 ? run_attend<T, 64, 1, MODE>(a, s) : run_attend<T, 64, 2, MODE>(a, s);
    return a.dv <= 64 ? run_attend<T, 128, 1, MODE>(a, s) : run_attend<T, 128, 2, MODE>(a, s);
}
template <typename T> hipError_t launch_attend(const AttendArgs& a, int mode, hipStream_t s) {
    switch (mode) {
        case kAttend: return pick_attend<T, kAttend>(a, s);
        case kDot: return pick_attend<T, kDot>(a, s);
        case kDotRows: return pick_attend<T, kDotRows>(a, s);
        default: return pick_attend<T, kLocal>(a, s);
    }
}

}  // namespace gdnl
