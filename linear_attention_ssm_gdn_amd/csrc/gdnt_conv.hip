// gdnt_conv.hip -- the backward pass of the causal depthwise conv (width 4)
// with SiLU.  With X the sequence's window and rows one after the other:
//   z_t = sum_j w_j X_{t-3+j},  dz_t = dy_t silu'(z_t),
//   dX_t = sum_j w_j dz_{t+3-j},  dw_j = sum_t dz_t X_{t-3+j}.
//
// A tile is 256 packed rows by 64 channels: 16 lanes side by side hold four
// channels each, 16 row groups hold 16 consecutive rows each.  A thread walks
// its rows and the three behind them (their dz reach back into its rows)
// with the last four X and dz in registers; the rows before and behind come
// from the caches, where the neighbouring row groups read them too.
#include "gdnt_device.hpp"

namespace gdnt {

constexpr int CR = 16;              // rows of a thread
constexpr int kConvThreads = 256;
constexpr int kConvWaves = kConvThreads / 64;
static_assert(kConvThreads / 16 * CR == kTileRows && 16 * 4 == kTileCols, "tile shape");

template <typename T, typename YT, bool VEC>
__global__ __launch_bounds__(kConvThreads) void k_conv_backward(const ConvBwdArgs A, int n_cols) {
    __shared__ float s_w[kConvWaves][4][kTileCols];
    const int64_t tile = blockIdx.x / n_cols;
    const int col = (int)(blockIdx.x % n_cols);
    const int lane = threadIdx.x & 63, cl = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t Cp = (int64_t)n_cols * kTileCols;
    const int64_t r0 = tile * kTileRows + rg * CR, c0 = (int64_t)col * kTileCols + cl * 4;
    const int64_t left = (int64_t)A.C - c0;
    const int nc = left >= 4 ? 4 : left > 0 ? (int)left : 0;

    // row map of r0-3 .. r0+CR+2 (entry k is row r0-3+k); the map is padded
    // to whole tiles, rows outside it belong to nothing
    int32_t m[CR + 6];
    const int64_t n_map = (A.n_rows + kTileRows - 1) / kTileRows * kTileRows;
#pragma unroll
    for (int k = 0; k < CR + 6; ++k) {
        const int64_t r = r0 - 3 + k;
        m[k] = r >= 0 && r < n_map ? A.map[r] : -1;
    }
    float wt[4][4];  // [tap][channel]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) wt[j][i] = i < nc ? to_f32(static_cast<const T*>(A.conv_w)[(c0 + i) * 4 + j]) : 0.0f;

    const T* px = static_cast<const T*>(A.x) + c0;
    const YT* py = static_cast<const YT*>(A.dy) + c0;
    T* pdx = static_cast<T*>(A.dx) + c0;
    Raw4<T> rx[CR + 6];
    Raw4<YT> ry[CR + 3];
#pragma unroll
    for (int k = 0; k < CR + 6; ++k) {
        rx[k] = zero4<T>();
        if (m[k] >= 0 && nc > 0) rx[k] = load4<T, VEC>(px + (r0 - 3 + k) * A.x_stride, nc);
    }
#pragma unroll
    for (int k = 0; k < CR + 3; ++k) {
        ry[k] = zero4<YT>();
        if (m[k + 3] >= 0 && nc > 0) ry[k] = load4<YT, VEC>(py + (r0 + k) * A.dy_stride, nc);
    }

    // X of the three rows before the current one, dz of the last four rows
    float X[3][4], dz[4][4], dw[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) { dz[j][i] = 0.0f; dw[j][i] = 0.0f; }

    // before row r0: where it continues a sequence, the rows above it that do
    // too; further up, the sequence's window
    auto window = [&](int32_t mr, int row, float (&v)[4]) {
        const int seq = mr >> 2;
        const bool init = A.window && (A.has_init ? A.has_init[seq] != 0 : true);
        const int64_t at = init ? (int64_t)A.page_idx[seq] * A.window_stride + row * (int64_t)A.C + c0 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = init && i < nc ? to_f32(static_cast<const T*>(A.window)[at + i]) : 0.0f;
    };
    {
        int have = 0;  // rows above r0 of the same sequence, at most 3
        if (m[3] >= 0 && !(m[3] & 1)) have = (m[2] & 1) ? 1 : (m[1] & 1) ? 2 : 3;
#pragma unroll
        for (int j = 0; j < 3; ++j) {  // X[j] is row r0 - 3 + j
#pragma unroll
            for (int i = 0; i < 4; ++i) X[j][i] = rx[j].get(i);
            if (m[3] >= 0 && j < 3 - have) window(m[3], j + have, X[j]);
        }
    }
#pragma unroll
    for (int k = 0; k < CR + 3; ++k) {  // row r0 + k
        const int32_t mr = m[k + 3];
        const bool in = mr >= 0, first = in && (mr & 1);
        if (k > 0 && first) {
#pragma unroll
            for (int j = 0; j < 3; ++j) window(mr, j, X[j]);
        }
        float x0[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x0[i] = rx[k + 3].get(i);
            float g = ry[k].get(i);
            if (A.activation) {
                const float z = fmaf(wt[3][i], x0[i], fmaf(wt[2][i], X[2][i], fmaf(wt[1][i], X[1][i], wt[0][i] * X[0][i])));
                const float sg = sigmoid_hw(z);
                g *= sg * fmaf(z, 1.0f - sg, 1.0f);
            }
            dz[0][i] = dz[1][i]; dz[1][i] = dz[2][i]; dz[2][i] = dz[3][i];
            dz[3][i] = in ? g : 0.0f;
        }
        if (k < CR) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dw[0][i] = fmaf(dz[3][i], X[0][i], dw[0][i]);
                dw[1][i] = fmaf(dz[3][i], X[1][i], dw[1][i]);
                dw[2][i] = fmaf(dz[3][i], X[2][i], dw[2][i]);
                dw[3][i] = fmaf(dz[3][i], x0[i], dw[3][i]);
            }
        }
        if (k >= 3) {  // dX of row p = r0 + k - 3, whose dz is dz[0]
            const int32_t m0 = m[k], m1 = m[k + 1], m2 = m[k + 2];
            // how many rows of the sequence follow row p, at most 3
            const int after = (m0 & 2) ? 0 : (m1 & 2) ? 1 : (m2 & 2) ? 2 : 3;
            if (m0 >= 0) {
                float dx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    dx[i] = wt[3][i] * dz[0][i];
                    if (after >= 1) dx[i] = fmaf(wt[2][i], dz[1][i], dx[i]);
                    if (after >= 2) dx[i] = fmaf(wt[1][i], dz[2][i], dx[i]);
                    if (after >= 3) dx[i] = fmaf(wt[0][i], dz[3][i], dx[i]);
                }
                if (after < 3 && A.d_window) {  // row p is row 2 - after of the rolled window
                    const float* p = A.d_window + ((int64_t)(m0 >> 2) * 3 + 2 - after) * A.C + c0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < nc) dx[i] += p[i];
                }
                if (nc > 0) store4<VEC>(pdx + (r0 + k - 3) * A.dx_stride, dx, nc);
                if ((m0 & 1) && A.d_window0) {
                    const int seq = m0 >> 2, T_ = after + 1;  // rows of the sequence, 4 for 4 and more
                    const bool init = A.window && (A.has_init ? A.has_init[seq] != 0 : true);
                    const float* src = A.d_window ? A.d_window + (int64_t)seq * 3 * A.C + c0 : nullptr;
                    float* dst = A.d_window0 + (int64_t)seq * 3 * A.C + c0;
#pragma unroll
                    for (int row = 0; row < 3; ++row)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float v = 0.0f;  // row `row` meets tap row - t of row t
#pragma unroll
                            for (int t = 0; t <= row; ++t)
                                if (t < T_) v = fmaf(wt[row - t][i], dz[t][i], v);
                            // still in the rolled window, T rows further up
                            if (row >= T_ && src && i < nc) v += src[(row - T_) * (int64_t)A.C + i];
                            if (i < nc) dst[row * (int64_t)A.C + i] = init ? v : 0.0f;
                        }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) { X[0][i] = X[1][i]; X[1][i] = X[2][i]; X[2][i] = x0[i]; }
    }
    // d_conv_w over the tile's rows: lanes, then waves
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

template <typename T, typename YT, bool VEC> static hipError_t conv_t(const ConvBwdArgs& a, hipStream_t s) {
    const int nc = (int)(padded_channels(a.C) / kTileCols);
    const int64_t nt = n_tiles(a.n_rows), grid = nt * nc;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    if (grid > 0)
        hipLaunchKernelGGL((k_conv_backward<T, YT, VEC>), dim3((unsigned)grid), dim3(kConvThreads), 0, s, a, nc);
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
