// gdnt_kernels.h -- argument blocks and launchers of the training-side
// operators (the C ABI in gdnt_api.cpp validates arguments and calls these).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct gdn_dims;

namespace gdn {
// The checks of gdn_api.cpp on gdn_dims (GDN_OK, GDN_ERR_ARG or GDN_ERR_UNSUPPORTED).
int32_t dims_status(const struct gdn_dims* d);
}  // namespace gdn

namespace gdnt {

constexpr int kTileRows = 256;  // packed rows of a tile: also the distance of the kept states
constexpr int kTileCols = 64;   // channels of a tile

// The row map: for each packed row -1 (no sequence, or a padding or skipped
// one) or sequence * 4 + 2 * (last row) + (first row).
struct MapArgs {
    const int32_t* cu; const int32_t* page_idx; int32_t n_seqs;
    int64_t n_rows, n_map;         // rows, and rows rounded up to the tile
    int32_t page_limit, max_len;   // 0 <= page < page_limit; max_len 0: any length
    int32_t* map;
    uint32_t* zero; int64_t n_zero;  // words to clear for the kernel that follows
    // a backward pass hands the final gradient of empty sequences through and
    // clears that of skipped ones: rows of `width` values, NULL src: zeros,
    // NULL dst: nothing to do
    const float* pass_src; float* pass_dst; int64_t pass_width;
    int32_t* err;
};

struct ScanArgs {
    const void* x; const void* a; const void* b; int64_t x_stride, ab_stride;
    int64_t n_rows;
    const int32_t* cu; const int32_t* page_idx; const uint8_t* has_init; int32_t n_seqs, max_len;
    const float* a_log; const float* dt_bias;
    const void* st_in; int64_t st_in_stride; void* st_out; int64_t st_out_stride; int32_t page_limit;
    void* h; int64_t h_stride;
    float* states;                       // kept states [n_tiles][C]
    int8_t* q; float* q_scale;           // 8-bit checkpoint
    // backward pass
    const void* dh; int64_t dh_stride; const float* d_state;
    void* dx; int64_t dx_stride; void* da; void* db; int64_t dab_stride;
    float* d_a_log; float* d_dt_bias; float* d_state0;
    // workspace
    int32_t* map; uint32_t* ticket; uint64_t* chain; float* part;
    int32_t C, act_dtype, state_dtype;
    bool vec;                            // every row starts aligned for 4-channel vectors and C % 4 == 0
    bool vec8;                           // backward: every row that is read starts on 16 bytes and C % 8 == 0
    int32_t* err;
};

struct ConvBwdArgs {
    const void* x; int64_t x_stride; const void* dy; int64_t dy_stride;
    int64_t n_rows;
    const int32_t* cu; const int32_t* page_idx; const uint8_t* has_init; int32_t n_seqs, max_len;
    const void* conv_w; const void* window; int64_t window_stride; int32_t page_limit;
    const float* d_window;
    void* dx; int64_t dx_stride; float* d_conv_w; float* d_window0;
    int32_t* map; float* part;
    int32_t C, activation, act_dtype, dy_dtype;
    bool vec;
    int32_t* err;
};

inline int64_t n_tiles(int64_t n_rows) { return (n_rows + kTileRows - 1) / kTileRows; }
__host__ __device__ inline int64_t padded_channels(int64_t C) { return (C + kTileCols - 1) / kTileCols * kTileCols; }

// Workgroups of the scan kernels, eight waves each; those of the forward pass
// (128 rows by 128 channels) and of the backward pass (256 by 64), the more of them.
constexpr int kScanThreads = 512;
inline int64_t scan_groups(int64_t n_rows, int64_t C) {
    const int64_t fwd = ((n_rows + 127) / 128) * ((C + 127) / 128);
    const int64_t bwd = n_tiles(n_rows) * (padded_channels(C) / kTileCols);
    return fwd > bwd ? fwd : bwd;
}
// Of the one-launch form: 256 threads, four channels each, to a sequence.
constexpr int kRowsThreads = 256;
inline int64_t scan_rows_groups(int64_t n_seqs, int64_t C) { return n_seqs * ((C + 4 * kRowsThreads - 1) / (4 * kRowsThreads)); }

// k_conv_backward: four strips to a workgroup, 256 channels wide.
constexpr int kConvWaves = 4;
constexpr int kConvCols = 256;
// Rows of a strip.  A strip reads six rows beside its own and computes three
// twice, so long strips cost least where there are enough of them, and the
// rows of one are walked one after the other: 57, 25, 13 rows take 374, 398,
// 474 us over 32768 x 8192 channels (18400 strips of 57), 55, 47, 54 us over
// 2159 x 8192 (1216, 2784, 5344 strips) and 54, 39, 31 us over 2066 x 672.
constexpr int kConvOwn[3] = {57, 25, 13};
// The fewest rows (of this many columns) for which there are enough strips of `own` rows.
inline int64_t conv_rows_from(int own, int64_t nc) { return ((2048 + nc - 1) / nc - 1) * own + 1; }
inline int conv_rows(int64_t n_rows, int64_t C) {
    const int64_t nc = (C + kConvCols - 1) / kConvCols;
    for (int i = 0; i < 2; ++i)
        if (n_rows >= conv_rows_from(kConvOwn[i], nc)) return kConvOwn[i];
    return kConvOwn[2];
}
inline int64_t conv_tiles(int64_t n_rows, int64_t C) {
    const int64_t rows = kConvWaves * conv_rows(n_rows, C);
    return (n_rows + rows - 1) / rows;
}
inline int64_t conv_groups(int64_t n_rows, int64_t C) {
    return conv_tiles(n_rows, C) * ((C + kConvCols - 1) / kConvCols);
}
// The most tiles that a batch of up to n_rows rows has: a batch just too small
// for longer strips has more of them than one just large enough.
inline int64_t conv_tiles_up_to(int64_t n_rows, int64_t C) {
    const int64_t nc = (C + kConvCols - 1) / kConvCols;
    int64_t most = conv_tiles(n_rows, C);
    for (int i = 0; i < 2; ++i) {
        const int64_t below = conv_rows_from(kConvOwn[i], nc) - 1;
        if (below < n_rows && conv_tiles(below, C) > most) most = conv_tiles(below, C);
    }
    return most;
}

hipError_t launch_map(const MapArgs& a, hipStream_t s);
hipError_t launch_scan_rows(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_forward(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s);
hipError_t launch_conv_backward(const ConvBwdArgs& a, hipStream_t s);
// out[j][c] = sum over tiles of part[tile][j][c], j < n_out, in fp64 and in tile order; out is
// out0 (j = 0), out1 (j = 1), or out0 [C][n_out] when out1 is NULL.
hipError_t launch_sum_tiles(const float* part, int64_t n_tiles, int32_t C, int n_out, float* out0, float* out1,
                            hipStream_t s);
// The row map of a scan call, and the words its kernels find at zero.
MapArgs scan_map_args(const ScanArgs& a);
// Chain words and partial sums of the scan's workspace (gdnt_api.cpp lays it out).
size_t scan_chain_bytes(int64_t n_rows, int32_t C);

}  // namespace gdnt
