// gdnt_conv.hip -- the backward pass of the causal depthwise conv (width 4)
// with SiLU.  With X the sequence's window and rows one after the other:
//   z_t = sum_j w_j X_{t-3+j},  dz_t = dy_t silu'(z_t),
//   dX_t = sum_j w_j dz_{t+3-j},  dw_j = sum_t dz_t X_{t-3+j}.
//
// A wave walks a strip of `own` rows by 256 channels, a lane four of them, and
// the three rows behind the strip, whose dz reach back into it: four rows at a
// time with the next four already loading.  Everything about a row is uniform
// over the wave, and a row's piece is 512 consecutive bytes in bf16 (a copy
// runs at 5.5 TB/s in such pieces here, at 4.7 in pieces of 128).  The rows
// around a strip come from the caches, where the neighbouring waves read them
// too.  Walking down, row t completes dX of row t-3 and adds to the three
// after it, so seen from row t there are three open sums.  The rows before a
// sequence's first are its window: their sums are d_window0, and where a
// sequence ends the open sums are the rows of its rolled window, where
// d_window joins.
//
// Bound by memory: 32768 x 8192 in bf16 takes 340 us for 1.61 GB (4.7 TB/s, 93%
// of a large copy's rate; 1.72 GB with what strips read twice, 5.0 TB/s) at 26
// vector instructions an element.  VEC (rows on four elements) takes 372 us a
// call there; others, through 64-bit addresses, 443 (fp32 662 and 790; 2159 rows
// in bf16 44 and 48).
#include "gdnt_device.hpp"

namespace gdnt {

constexpr int kConvThreads = kConvWaves * 64;

// The rows of one tensor around a wave's strip; row k counts from the strip's
// first, from -3 on.  VEC: a buffer descriptor, a scalar offset for the row
// (32 bits reach over 63 rows of up to 2^24 elements).
template <typename T, bool VEC> struct Strip {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t row, at;  // bytes
    T* p;
    int64_t stride;
    __device__ __forceinline__ Strip(const void* base, int64_t stride_, int64_t n_rows, int64_t r0, int32_t C,
                                     int64_t col, int lane)
        : row((uint32_t)stride_ * (uint32_t)sizeof(T)), at(lane * 4 * (uint32_t)sizeof(T)),
          p(static_cast<T*>(const_cast<void*>(base)) + (r0 - 3) * stride_ + col), stride(stride_) {
        if constexpr (VEC) {
            int64_t bytes = ((n_rows - 1 - (r0 - 3)) * stride_ + C - col) * (int64_t)sizeof(T);
            bytes = bytes < 0 ? 0 : bytes > 0xfffffffcll ? 0xfffffffcll : bytes;
            rs = __builtin_amdgcn_make_buffer_rsrc(p, 0, (uint32_t)bytes, 0x00020000);
        } else {
            p += lane * 4;
        }
    }
    __device__ __forceinline__ Raw4<T> load(int k, int nc) const {
        Raw4<T> v;
        if constexpr (VEC) {
            if constexpr (sizeof(T) == 2) v.v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rs, at, (uint32_t)(k + 3) * row, 0));
            else v.v = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, (uint32_t)(k + 3) * row, 0));
        } else {
            v = load4<T, false>(p + (k + 3) * stride, nc);
        }
        return v;
    }
    __device__ __forceinline__ void store(int k, int nc, const float (&f)[4]) const {
        if (nc == 0) return;
        if constexpr (VEC) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
            if constexpr (sizeof(T) == 2) {
                const u32x2 v = {gdn::f32x2_to_bf16x2(f[0], f[1]), gdn::f32x2_to_bf16x2(f[2], f[3])};
                __builtin_amdgcn_raw_buffer_store_b64(v, rs, at, (uint32_t)(k + 3) * row, 0);
            } else {
                const u32x4 v = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
                __builtin_amdgcn_raw_buffer_store_b128(v, rs, at, (uint32_t)(k + 3) * row, 0);
            }
        } else {
            store4<false>(p + (k + 3) * stride, f, nc);
        }
    }
};

template <typename T, typename YT> struct ConvRows {  // four rows as loaded
    Raw4<T> x[4];
    Raw4<YT> y[4];
};

template <typename T, typename YT, bool VEC>
__global__ __launch_bounds__(kConvThreads) void k_conv_backward(const ConvBwdArgs A, int n_cols, int own) {
    __shared__ float4 s_w[kConvWaves][4][64];
    const int64_t tile = blockIdx.x / n_cols;
    const int col = (int)(blockIdx.x % n_cols);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t r0 = (tile * kConvWaves + wave) * own, cb = (int64_t)col * kConvCols, c0 = cb + lane * 4;
    const int64_t left = (int64_t)A.C - c0;
    const int nc = left >= 4 ? 4 : left > 0 ? (int)left : 0;
    const int64_t n_map = (A.n_rows + kTileRows - 1) / kTileRows * kTileRows;

    // bit k + 3 stands for row r0 + k, k = -3 .. own + 2 < 61: is it a
    // sequence's, and is it not the successor of the row above it
    const int64_t rm = r0 - 3 + lane;
    const int32_t m = rm >= 0 && rm < n_map ? A.map[rm] : -1;
    const uint64_t in = __ballot(m >= 0), cut = __ballot(m < 0 || (m & 1));
    auto seq_of = [&](int k) { return __builtin_amdgcn_readlane(m, k + 3) >> 2; };

    float wt[4][4], dw[4][4];  // [tap][channel]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            wt[j][i] = i < nc ? to_f32(static_cast<const T*>(A.conv_w)[(c0 + i) * 4 + j]) : 0.0f;
            dw[j][i] = 0.0f;
        }

    const Strip<T, VEC> Xs(A.x, A.x_stride, A.n_rows, r0, A.C, cb, lane), Ds(A.dx, A.dx_stride, A.n_rows, r0, A.C, cb, lane);
    const Strip<YT, VEC> Ys(A.dy, A.dy_stride, A.n_rows, r0, A.C, cb, lane);

    auto has_init = [&](int seq) { return A.window && (A.has_init ? A.has_init[seq] != 0 : true); };
    auto window = [&](int seq, int row, float (&v)[4]) {
        const bool init = has_init(seq);
        const int64_t at = init ? (int64_t)A.page_idx[seq] * A.window_stride + row * (int64_t)A.C + c0 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = init && i < nc ? to_f32(static_cast<const T*>(A.window)[at + i]) : 0.0f;
    };
    auto put_window = [&](int seq, int row, const float (&v)[4]) {
        if (!A.d_window0) return;
        const bool init = has_init(seq);
        float* p = A.d_window0 + ((int64_t)seq * 3 + row) * A.C + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < nc) p[i] = init ? v[i] : 0.0f;
    };
    auto load = [&](ConvRows<T, YT>& g, int k) {  // rows r0 + k .. r0 + k + 3, k < own + 3
        const uint32_t have = (uint32_t)(in >> (k + 3)) & 15u;
        if (have == 15u && nc > 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g.x[e] = Xs.load(k + e, nc);
                g.y[e] = Ys.load(k + e, nc);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g.x[e] = zero4<T>();
                g.y[e] = zero4<YT>();
                if ((have >> e & 1u) && nc > 0) {
                    g.x[e] = Xs.load(k + e, nc);
                    g.y[e] = Ys.load(k + e, nc);
                }
            }
        }
    };

    // X of the three rows before the current one and the open sums of the same rows
    float X[3][4], acc[3][4] = {};
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        Raw4<T> v = zero4<T>();
        if ((in >> j & 1) && nc > 0) v = Xs.load(j - 3, nc);
#pragma unroll
        for (int i = 0; i < 4; ++i) X[j][i] = v.get(i);
    }
    if ((in >> 3 & 1) && !(cut >> 3 & 1) && (cut >> 1 & 3)) {  // a sequence begins one or two rows above r0
        const int have = (cut >> 2 & 1) ? 1 : 2, seq = seq_of(0);
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < 3 - have) window(seq, j + have, X[j]);
    }

    bool open = true;  // rows of this strip, or behind them with their sums open, are left
    auto rows4 = [&](const ConvRows<T, YT>& g, int k0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = k0 + e;
            // the rows k, k - 1, k - 2 and whether a sequence begins there
            const uint32_t near = (uint32_t)(cut >> (k + 1)) & 7u;
            if (near & 4u) {
                if (k > 0 && open && (in >> (k + 2) & 1)) {  // row k - 1 ended its sequence
                    const int seq = seq_of(k - 1);
                    // bit d: a sequence begins at row k - 1 - d
                    const uint32_t begins = ((near >> 1 & 1u) | (near << 1 & 2u));
                    const int rows = (begins & 1u) ? 1 : (begins & 2u) ? 2 : 3;  // of the sequence, 3: or more
#pragma unroll
                    for (int j = 0; j < 3; ++j) {
                        const int p = k - 3 + j;  // the row this sum belongs to, if it is one
                        if (A.d_window) {
                            const float* src = A.d_window + ((int64_t)seq * 3 + j) * A.C + c0;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (i < nc) acc[j][i] += src[i];
                        }
                        if (j >= 3 - rows) {
                            if (p >= 0 && p < own) Ds.store(p, nc, acc[j]);
                        } else if (k - rows >= 0) {  // the sequence begins in this strip
                            put_window(seq, rows + j, acc[j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 3; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
                open = open && k < own;  // the rest is the next strip's
                const bool begins = open && (in >> (k + 3) & 1);
                const int seq = begins ? seq_of(k) : 0;
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    if (begins) window(seq, j, X[j]);
                    else X[j][0] = X[j][1] = X[j][2] = X[j][3] = 0.0f;  // a row of no sequence adds nothing
                }
            }
            float out[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x0 = g.x[e].get(i);
                float dz = g.y[e].get(i);
                if (A.activation) {
                    const float z = fmaf(wt[3][i], x0, fmaf(wt[2][i], X[2][i], fmaf(wt[1][i], X[1][i], wt[0][i] * X[0][i])));
                    const float sg = sigmoid_hw(z);
                    dz *= sg * fmaf(z, 1.0f - sg, 1.0f);
                }
                if (k < own) {
                    dw[0][i] = fmaf(dz, X[0][i], dw[0][i]);
                    dw[1][i] = fmaf(dz, X[1][i], dw[1][i]);
                    dw[2][i] = fmaf(dz, X[2][i], dw[2][i]);
                    dw[3][i] = fmaf(dz, x0, dw[3][i]);
                }
                out[i] = fmaf(wt[0][i], dz, acc[0][i]);
                acc[0][i] = fmaf(wt[1][i], dz, acc[1][i]);
                acc[1][i] = fmaf(wt[2][i], dz, acc[2][i]);
                acc[2][i] = wt[3][i] * dz;
                X[0][i] = X[1][i]; X[1][i] = X[2][i]; X[2][i] = x0;
            }
            if (near == 0) {
                if (k >= 3 && open) Ds.store(k - 3, nc, out);
            } else if (open && (in >> (k + 3) & 1)) {
                const int t = (near & 4u) ? 0 : (near & 2u) ? 1 : 2;  // row of its sequence: completes window row t
                if (k - t >= 0) put_window(seq_of(k), t, out);
            }
        }
    };
    // two buffers that change roles; own + 3 is a multiple of 4
    ConvRows<T, YT> ga, gb;
    load(ga, 0);
    for (int k0 = 0; k0 < own + 3; k0 += 8) {
        if (k0 + 4 < own + 3) load(gb, k0 + 4);
        rows4(ga, k0);
        if (k0 + 4 >= own + 3) break;
        if (k0 + 8 < own + 3) load(ga, k0 + 8);
        rows4(gb, k0 + 4);
    }
    // d_conv_w over the workgroup's strips
#pragma unroll
    for (int j = 0; j < 4; ++j) s_w[wave][j][lane] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
    __syncthreads();
    const int64_t Cp = padded_channels(A.C);
    if (c0 < Cp) {  // tap `wave`
        const float4 p = s_w[0][wave][lane], q = s_w[1][wave][lane], r = s_w[2][wave][lane], s = s_w[3][wave][lane];
        *reinterpret_cast<float4*>(A.part + (tile * 4 + wave) * Cp + c0) =
            make_float4((p.x + q.x) + (r.x + s.x), (p.y + q.y) + (r.y + s.y), (p.z + q.z) + (r.z + s.z),
                        (p.w + q.w) + (r.w + s.w));
    }
}

template <typename T, typename YT, bool VEC> static hipError_t conv_t(const ConvBwdArgs& a, hipStream_t s) {
    const int nc = (int)((a.C + kConvCols - 1) / kConvCols);
    const int own = conv_rows(a.n_rows, a.C);
    const int64_t nt = conv_tiles(a.n_rows, a.C), grid = nt * nc;
    if (grid > 0) {
        hipLaunchKernelGGL((k_conv_backward<T, YT, VEC>), dim3((unsigned)grid), dim3(kConvThreads), 0, s, a, nc, own);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_sum_tiles(a.part, nt, a.C, 4, a.d_conv_w, nullptr, s);
}

template <typename T, typename YT> static hipError_t conv_v(const ConvBwdArgs& a, hipStream_t s) {
    return a.vec ? conv_t<T, YT, true>(a, s) : conv_t<T, YT, false>(a, s);
}

hipError_t launch_conv_backward(const ConvBwdArgs& a, hipStream_t s) {
    MapArgs m{};
    m.cu = a.cu; m.page_idx = a.page_idx; m.n_seqs = a.n_seqs;
    m.n_rows = a.n_rows; m.n_map = n_tiles(a.n_rows) * kTileRows;
    m.page_limit = a.page_limit; m.max_len = a.max_len; m.map = a.map; m.err = a.err;
    m.pass_src = a.d_window; m.pass_dst = a.d_window0; m.pass_width = (int64_t)3 * a.C;
    const hipError_t e = launch_map(m, s);
    if (e != hipSuccess) return e;
    if (a.act_dtype == GDN_BF16)
        return a.dy_dtype == GDN_BF16 ? conv_v<bf16_t, bf16_t>(a, s) : conv_v<bf16_t, float>(a, s);
    return a.dy_dtype == GDN_BF16 ? conv_v<float, bf16_t>(a, s) : conv_v<float, float>(a, s);
}

}  // namespace gdnt
