// gdnt_conv.hip -- the backward pass of the causal depthwise conv (width 4)
// with SiLU.  With X the sequence's window and rows one after the other:
//   z_t = sum_j w_j X_{t-3+j},  dz_t = dy_t silu'(z_t),
//   dX_t = sum_j w_j dz_{t+3-j},  dw_j = sum_t dz_t X_{t-3+j}.
//
// Sixteen lanes side by side hold four channels each, sixteen row groups of a
// workgroup hold `own` consecutive rows each.  A thread walks its rows and the
// three behind them, whose dz reach back into its rows, four rows at a time
// with the next four already loading; the rows around its own come from the
// caches, where the neighbouring row groups read them too.  Walking down, row
// t completes dX of row t-3 and adds to the three after it, so seen from row
// t there are three open sums.  The rows before a sequence's first are its
// window: their sums are d_window0, and where a sequence ends the open sums
// are the rows of its rolled window, where d_window joins.
#include <type_traits>

#include "gdnt_device.hpp"

namespace gdnt {

constexpr int kConvThreads = 256;
constexpr int kConvWaves = kConvThreads / 64;
constexpr int kConvGroups = kConvThreads / 16;

template <typename T, typename YT> struct ConvRows {  // four rows as loaded
    Raw4<T> x[4];
    Raw4<YT> y[4];
};

template <typename T, typename YT, bool VEC>
__global__ __launch_bounds__(kConvThreads) void k_conv_backward(const ConvBwdArgs A, int n_cols, int own) {
    __shared__ float s_w[kConvWaves][4][kTileCols];
    const int64_t tile = blockIdx.x / n_cols;
    const int col = (int)(blockIdx.x % n_cols);
    const int lane = threadIdx.x & 63, cl = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t Cp = (int64_t)n_cols * kTileCols;
    const int64_t r0 = (tile * kConvGroups + rg) * own, c0 = (int64_t)col * kTileCols + cl * 4;
    const int64_t left = (int64_t)A.C - c0;
    const int nc = left >= 4 ? 4 : left > 0 ? (int)left : 0;
    const int64_t n_map = (A.n_rows + kTileRows - 1) / kTileRows * kTileRows;

    // bit k + 3 stands for row r0 + k, k = -3 .. own + 2 < 61: is it a
    // sequence's, and is it not the successor of the row above it
    uint64_t in = 0, cut = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t r = r0 - 3 + q * 16 + cl;
        const int32_t m = r >= 0 && r < n_map ? A.map[r] : -1;
        in |= ((__ballot(m >= 0) >> (lane & 48)) & 0xffffull) << (q * 16);
        cut |= ((__ballot(m < 0 || (m & 1)) >> (lane & 48)) & 0xffffull) << (q * 16);
    }

    float wt[4][4], dw[4][4];  // [tap][channel]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            wt[j][i] = i < nc ? to_f32(static_cast<const T*>(A.conv_w)[(c0 + i) * 4 + j]) : 0.0f;
            dw[j][i] = 0.0f;
        }

    // Byte offsets from three rows above the workgroup's first: they fit 32 bits
    // where VEC is set (the launcher's rule on strides), which leaves one add a row.
    using Off = typename std::conditional<VEC, uint32_t, int64_t>::type;
    const int64_t t0 = tile * kConvGroups * own - 3;
    const int64_t cb = (int64_t)col * kTileCols;
    const char* px = static_cast<const char*>(A.x) + (t0 * A.x_stride + cb) * (int64_t)sizeof(T);
    const char* py = static_cast<const char*>(A.dy) + (t0 * A.dy_stride + cb) * (int64_t)sizeof(YT);
    char* pdx = static_cast<char*>(A.dx) + (t0 * A.dx_stride + cb) * (int64_t)sizeof(T);
    const Off sx = (Off)A.x_stride * (Off)sizeof(T), sy = (Off)A.dy_stride * (Off)sizeof(YT);
    const Off sd = (Off)A.dx_stride * (Off)sizeof(T);
    const Off row3 = (Off)(rg * own + 3);  // row r0 counted from t0
    const Off cx = (Off)(cl * 4 * sizeof(T)), cy = (Off)(cl * 4 * sizeof(YT));
    Off ox = row3 * sx + cx, oy = row3 * sy + cy, od = (row3 - 3) * sd + cx;  // rows to load, row to store
    auto at_x = [&](Off o) { return reinterpret_cast<const T*>(px + o); };
    auto at_y = [&](Off o) { return reinterpret_cast<const YT*>(py + o); };
    auto at_dx = [&](Off o) { return reinterpret_cast<T*>(pdx + o); };

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
                g.x[e] = load4<T, VEC>(at_x(ox + e * sx), nc);
                g.y[e] = load4<YT, VEC>(at_y(oy + e * sy), nc);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g.x[e] = zero4<T>();
                g.y[e] = zero4<YT>();
                if ((have >> e & 1u) && nc > 0) {
                    g.x[e] = load4<T, VEC>(at_x(ox + e * sx), nc);
                    g.y[e] = load4<YT, VEC>(at_y(oy + e * sy), nc);
                }
            }
        }
        ox += 4 * sx;
        oy += 4 * sy;
    };

    // X of the three rows before the current one and the open sums of the same rows
    float X[3][4], acc[3][4] = {};
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        Raw4<T> v = zero4<T>();
        if ((in >> j & 1) && nc > 0) v = load4<T, VEC>(at_x((row3 + j - 3) * sx + cx), nc);
#pragma unroll
        for (int i = 0; i < 4; ++i) X[j][i] = v.get(i);
    }
    if ((in >> 3 & 1) && !(cut >> 3 & 1) && (cut >> 1 & 3)) {  // a sequence begins one or two rows above r0
        const int have = (cut >> 2 & 1) ? 1 : 2, seq = A.map[r0] >> 2;
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < 3 - have) window(seq, j + have, X[j]);
    }

    bool open = true;  // rows of this thread, or behind them with their sums open, are left
    auto rows4 = [&](const ConvRows<T, YT>& g, int k0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = k0 + e;
            // the rows k, k - 1, k - 2 and whether a sequence begins there
            const uint32_t near = (uint32_t)(cut >> (k + 1)) & 7u;
            if (near & 4u) {
                if (k > 0 && open && (in >> (k + 2) & 1)) {  // row k - 1 ended its sequence
                    const int seq = A.map[r0 + k - 1] >> 2;
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
                            if (p >= 0 && p < own && nc > 0) store4<VEC>(at_dx((row3 + p) * sd + cx), acc[j], nc);
                        } else if (k - rows >= 0) {  // the sequence begins in this thread's rows
                            put_window(seq, rows + j, acc[j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 3; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
                open = open && k < own;  // the rest is the next thread's
                const bool begins = open && (in >> (k + 3) & 1);
                const int seq = begins ? A.map[r0 + k] >> 2 : 0;
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
                if (k >= 3 && open && nc > 0) store4<VEC>(at_dx(od), out, nc);
            } else if (open && (in >> (k + 3) & 1)) {
                const int t = (near & 4u) ? 0 : (near & 2u) ? 1 : 2;  // row of its sequence: completes window row t
                if (k - t >= 0) put_window(A.map[r0 + k] >> 2, t, out);
            }
            od += sd;
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
    // d_conv_w over the workgroup's rows: lanes, then waves
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = dw[j][i];
            v += __shfl_xor(v, 16);
            v += __shfl_xor(v, 32);
            if (lane < 16) s_w[wave][j][cl * 4 + i] = v;
        }
    __syncthreads();
    const int j = threadIdx.x >> 6, ch = lane;  // 4 taps by 64 channels
    A.part[(tile * 4 + j) * Cp + (int64_t)col * kTileCols + ch] =
        (s_w[0][j][ch] + s_w[1][j][ch]) + (s_w[2][j][ch] + s_w[3][j][ch]);
}

static int conv_rows(int64_t n_rows, int64_t C) {
    const int64_t nc = padded_channels(C) / kTileCols;
    return (n_rows + kConvGroups * 57 - 1) / (kConvGroups * 57) * nc >= 1024 ? 57 : 13;
}

template <typename T, typename YT, bool VEC> static hipError_t conv_t(const ConvBwdArgs& a, hipStream_t s) {
    const int nc = (int)(padded_channels(a.C) / kTileCols);
    // VEC addresses a workgroup's rows (16 * 57 + 6 at most) by 32-bit byte offsets
    if (VEC && (a.x_stride | a.dy_stride | a.dx_stride) >> 20) return conv_t<T, YT, false>(a, s);
    // 57 rows a thread where that leaves work for every compute unit, else 13
    const int own = conv_rows(a.n_rows, a.C);
    const int64_t nt = (a.n_rows + kConvGroups * own - 1) / (kConvGroups * own), grid = nt * nc;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    if (grid > 0)
        hipLaunchKernelGGL((k_conv_backward<T, YT, VEC>), dim3((unsigned)grid), dim3(kConvThreads), 0, s, a, nc, own);
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
