// gdnt_api.cpp -- the C ABI of include/gdn_train.h: argument validation,
// workspace layout and kernel launches.  As in gdn_api.cpp every check runs
// on the host before anything is launched.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gdn_train.h"
#include "gdnt_kernels.h"

#define GDN_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

using gdnt::n_tiles;
using gdnt::padded_channels;

// Batches of at most kRowsSeqs sequences whose longest has at most kRowsMax
// rows, and that keep nothing for a backward pass, run without a row map (one
// launch).  Over 4096 bf16 channels the one launch takes 19 us where the
// tiles take 28 (64 sequences of one row), 47 against 71 (1024 of 8), 230
// against 258 (4096 of 8); each of its workgroups looks over the bounds of
// every sequence before its own, so with 16384 of 8 it loses, 1188 against 956.
constexpr int32_t kRowsMax = 8, kRowsSeqs = 4096;

int64_t elem_size(int32_t dt) { return dt == GDN_BF16 ? 2 : 4; }
bool dtype_ok(int32_t dt) { return dt == GDN_F32 || dt == GDN_BF16; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int32_t from_hip(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }
size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

// Rows that start on their element's boundary, and on a 4-channel vector's
// (the one-launch form takes 62 us over 1024 x 8 rows of 4096 bf16 channels on
// the latter, 70 elsewhere; 64 rows take a launch's time either way).
bool rows_ok(const void* p, int64_t stride, int64_t C, int32_t dt) {
    // a wave's rows are addressed by 32-bit byte offsets
    return p && stride >= C && stride <= (1 << 24) && aligned(p, (size_t)elem_size(dt));
}
bool rows_vec(const void* p, int64_t stride, int32_t dt) {
    return stride % 4 == 0 && aligned(p, (size_t)(4 * elem_size(dt)));
}
int32_t check_dims(const gdnt_scan_dims* d) {
    if (!d || d->channels <= 0 || d->channels > (1 << 24)) return GDN_ERR_ARG;
    if (!dtype_ok(d->act_dtype) || !dtype_ok(d->state_dtype)) return GDN_ERR_ARG;
    return GDN_OK;
}

int32_t check_batch(const gdn_batch* b) {
    if (!b || b->n_seqs < 0 || b->max_seqlen < 0 || b->n_rows < 0) return GDN_ERR_ARG;
    // the row map holds 4 * sequence + 2 bits
    if (b->n_rows > INT32_MAX - 2 * gdnt::kTileRows || b->n_seqs > (1 << 29) - 1) return GDN_ERR_ARG;
    if (b->n_seqs > 0 && (!b->cu_seqlens || !b->page_idx)) return GDN_ERR_ARG;
    return GDN_OK;
}

// HIP launches fewer than 2^32 threads in a dimension.
int32_t check_launch(int64_t groups, int64_t threads) {
    return groups <= (int64_t)UINT32_MAX / threads ? GDN_OK : GDN_ERR_ARG;
}
int32_t check_rows(int64_t n_rows) {
    return n_rows >= 0 && n_rows <= INT32_MAX - 2 * gdnt::kTileRows ? GDN_OK : GDN_ERR_ARG;
}
int32_t check_scan_size(int64_t n_rows, int64_t C) {
    const int32_t st = check_rows(n_rows);
    return st != GDN_OK ? st : check_launch(gdnt::scan_groups(n_rows, C), gdnt::kScanThreads);
}
int32_t check_conv_size(int64_t n_rows, int64_t C) {
    const int32_t st = check_rows(n_rows);
    return st != GDN_OK ? st : check_launch(gdnt::conv_groups(n_rows, C), gdnt::kConvWaves * 64);
}

int32_t check_pool(const gdnt_scan_dims* d, const gdn_state_pool& s) {
    if (!s.base || s.n_pages < 0 || s.page_stride < d->channels) return GDN_ERR_ARG;
    return aligned(s.base, (size_t)elem_size(d->state_dtype)) ? GDN_OK : GDN_ERR_ARG;
}

// Scan workspace: row map, ticket (256 bytes), chain words, partial sums.
struct ScanWs {
    size_t ticket, chain, part, total;
};
ScanWs scan_ws(int64_t n_rows, int64_t C) {
    ScanWs w;
    const int64_t nt = n_tiles(n_rows);
    w.ticket = (size_t)nt * gdnt::kTileRows * sizeof(int32_t);
    w.chain = w.ticket + 256;
    w.part = round_up(w.chain + gdnt::scan_chain_bytes(n_rows, (int32_t)C));
    w.total = round_up(w.part + (size_t)nt * 2 * (size_t)padded_channels(C) * sizeof(float));
    return w;
}

// Conv workspace: row map, partial sums of `tiles` tiles.
size_t conv_ws(int64_t n_rows, int64_t C, int64_t tiles) {
    return round_up((size_t)n_tiles(n_rows) * gdnt::kTileRows * sizeof(int32_t) +
                    (size_t)tiles * 4 * (size_t)padded_channels(C) * sizeof(float));
}

size_t states_bytes(int64_t n_rows, int64_t C) { return (size_t)n_tiles(n_rows) * (size_t)C * sizeof(float); }
int64_t ckpt_blocks(int64_t n_rows, int64_t C) {
    return (n_rows + GDNT_CKPT_ROWS - 1) / GDNT_CKPT_ROWS * 3 * (padded_channels(C) / GDNT_CKPT_CHANNELS);
}

void set_ckpt(gdnt::ScanArgs& A, const void* ckpt) {
    A.q = static_cast<int8_t*>(const_cast<void*>(ckpt));
    A.q_scale = reinterpret_cast<float*>(A.q + ckpt_blocks(A.n_rows, A.C) * GDNT_CKPT_ROWS * GDNT_CKPT_CHANNELS);
}

gdnt::ScanArgs scan_args(const gdnt_scan_dims* d, const gdnt_scan_params* p, const gdn_batch* b,
                         const gdn_state_pool& in, void* ws, int32_t* err) {
    gdnt::ScanArgs A{};
    A.n_rows = b->n_rows; A.cu = b->cu_seqlens; A.page_idx = b->page_idx; A.has_init = b->has_init;
    A.n_seqs = b->n_seqs; A.max_len = b->max_seqlen;
    A.a_log = p->a_log; A.dt_bias = p->dt_bias;
    A.st_in = in.base; A.st_in_stride = in.page_stride; A.page_limit = in.n_pages;
    A.C = d->channels; A.act_dtype = d->act_dtype; A.state_dtype = d->state_dtype; A.err = err;
    char* base = static_cast<char*>(ws);
    const ScanWs w = scan_ws(b->n_rows, d->channels);
    A.map = reinterpret_cast<int32_t*>(base);
    A.ticket = reinterpret_cast<uint32_t*>(base + w.ticket);
    A.chain = reinterpret_cast<uint64_t*>(base + w.chain);
    A.part = reinterpret_cast<float*>(base + w.part);
    return A;
}

}  // namespace

GDN_EXPORT int32_t gdnt_scan_workspace_bytes(const gdnt_scan_dims* dims, int32_t n_seqs, int64_t n_rows,
                                             size_t* out_bytes) {
    int32_t st;
    if ((st = check_dims(dims)) != GDN_OK) return st;
    if (!out_bytes || n_seqs < 0) return GDN_ERR_ARG;
    if ((st = check_scan_size(n_rows, dims->channels)) != GDN_OK) return st;
    *out_bytes = scan_ws(n_rows, dims->channels).total;
    return GDN_OK;
}

GDN_EXPORT int32_t gdnt_scan_saved_bytes(const gdnt_scan_dims* dims, int64_t n_rows, size_t* states, size_t* ckpt) {
    int32_t st;
    if ((st = check_dims(dims)) != GDN_OK) return st;
    if ((st = check_scan_size(n_rows, dims->channels)) != GDN_OK) return st;
    if (states) *states = states_bytes(n_rows, dims->channels);
    if (ckpt) *ckpt = (size_t)ckpt_blocks(n_rows, dims->channels) * (GDNT_CKPT_ROWS * GDNT_CKPT_CHANNELS + sizeof(float));
    return GDN_OK;
}

GDN_EXPORT int32_t gdnt_conv_workspace_bytes(const gdn_dims* dims, int32_t n_seqs, int64_t n_rows,
                                             size_t* out_bytes) {
    int32_t st;
    if ((st = gdn::dims_status(dims)) != GDN_OK) return st;
    if (!out_bytes || n_seqs < 0) return GDN_ERR_ARG;
    const int64_t C = 2 * (int64_t)dims->h_k * dims->d_k + (int64_t)dims->h_v * dims->d_v;
    if ((st = check_conv_size(n_rows, C)) != GDN_OK) return st;
    *out_bytes = conv_ws(n_rows, C, gdnt::conv_tiles_up_to(n_rows, C));
    return GDN_OK;
}

GDN_EXPORT int32_t gdnt_scan_forward(const gdnt_scan_dims* dims, const gdnt_scan_params* params, const void* x,
                                     int64_t x_stride, const void* a, const void* b, int64_t ab_stride,
                                     const gdn_batch* batch, gdn_state_pool state_in, gdn_state_pool state_out,
                                     void* h, int64_t h_stride, float* states, void* ckpt, void* workspace,
                                     size_t ws_bytes, int32_t* err, void* stream) {
    int32_t st;
    if ((st = check_dims(dims)) != GDN_OK) return st;
    if (!params || !params->a_log || !params->dt_bias) return GDN_ERR_ARG;
    if ((st = check_batch(batch)) != GDN_OK) return st;
    if ((st = check_scan_size(batch->n_rows, dims->channels)) != GDN_OK) return st;
    if (ckpt && (!states || !aligned(ckpt, 256))) return GDN_ERR_ARG;
    if (states && !aligned(states, 16)) return GDN_ERR_ARG;
    if (batch->n_seqs == 0) return GDN_OK;
    if ((st = check_pool(dims, state_in)) != GDN_OK || (st = check_pool(dims, state_out)) != GDN_OK) return st;
    const int64_t C = dims->channels;
    const int32_t dt = dims->act_dtype, sdt = dims->state_dtype;
    if (batch->n_rows > 0 && (!rows_ok(x, x_stride, C, dt) || !rows_ok(a, ab_stride, C, dt) ||
                              !rows_ok(b, ab_stride, C, dt) || !rows_ok(h, h_stride, C, dt)))
        return GDN_ERR_ARG;
    const bool rows = batch->max_seqlen > 0 && batch->max_seqlen <= kRowsMax && batch->n_seqs <= kRowsSeqs && !states;
    if (rows && (st = check_launch(gdnt::scan_rows_groups(batch->n_seqs, C), gdnt::kRowsThreads)) != GDN_OK) return st;
    if (!rows && (ws_bytes < scan_ws(batch->n_rows, C).total || !workspace || !aligned(workspace, 256)))
        return GDN_ERR_ARG;
    gdnt::ScanArgs A = scan_args(dims, params, batch, state_in, workspace, err);
    A.x = x; A.a = a; A.b = b; A.x_stride = x_stride; A.ab_stride = ab_stride;
    A.st_out = state_out.base; A.st_out_stride = state_out.page_stride;
    if (state_out.n_pages < A.page_limit) A.page_limit = state_out.n_pages;
    A.h = h; A.h_stride = h_stride; A.states = states;
    if (ckpt) set_ckpt(A, ckpt);
    A.vec = C % 4 == 0 && rows_vec(x, x_stride, dt) && rows_vec(a, ab_stride, dt) && rows_vec(b, ab_stride, dt) &&
            rows_vec(h, h_stride, dt) && rows_vec(state_in.base, state_in.page_stride, sdt) &&
            rows_vec(state_out.base, state_out.page_stride, sdt);
    return from_hip(rows ? gdnt::launch_scan_rows(A, (hipStream_t)stream)
                         : gdnt::launch_scan_forward(A, (hipStream_t)stream));
}

GDN_EXPORT int32_t gdnt_scan_backward(const gdnt_scan_dims* dims, const gdnt_scan_params* params, const void* x,
                                      int64_t x_stride, const void* a, const void* b, int64_t ab_stride,
                                      const void* ckpt, const gdn_batch* batch, gdn_state_pool state_in,
                                      const float* states, const void* dh, int64_t dh_stride, const float* d_state,
                                      void* dx, int64_t dx_stride, void* da, void* db, int64_t dab_stride,
                                      float* d_a_log, float* d_dt_bias, float* d_state0, void* workspace,
                                      size_t ws_bytes, int32_t* err, void* stream) {
    int32_t st;
    if ((st = check_dims(dims)) != GDN_OK) return st;
    if (!params || !params->a_log || !params->dt_bias || !d_a_log || !d_dt_bias) return GDN_ERR_ARG;
    if ((st = check_batch(batch)) != GDN_OK) return st;
    if ((st = check_scan_size(batch->n_rows, dims->channels)) != GDN_OK) return st;
    gdn_batch bt = *batch;
    if (bt.n_seqs == 0) bt.n_rows = 0;  // no row belongs to a sequence
    const int64_t C = dims->channels;
    const int32_t dt = dims->act_dtype;
    if (bt.n_seqs > 0 && (st = check_pool(dims, state_in)) != GDN_OK) return st;
    if (ckpt && (x || a || b || !aligned(ckpt, 256))) return GDN_ERR_ARG;
    if (bt.n_rows > 0) {
        if (!ckpt && (!rows_ok(x, x_stride, C, dt) || !rows_ok(a, ab_stride, C, dt) || !rows_ok(b, ab_stride, C, dt)))
            return GDN_ERR_ARG;
        if (!rows_ok(dh, dh_stride, C, dt) || !rows_ok(dx, dx_stride, C, dt) || !rows_ok(da, dab_stride, C, dt) ||
            !rows_ok(db, dab_stride, C, dt))
            return GDN_ERR_ARG;
        if (!states || !aligned(states, 16)) return GDN_ERR_ARG;
    }
    if (ws_bytes < scan_ws(bt.n_rows, C).total || !workspace || !aligned(workspace, 256)) return GDN_ERR_ARG;
    gdnt::ScanArgs A = scan_args(dims, params, &bt, state_in, workspace, err);
    A.x = x; A.a = a; A.b = b; A.x_stride = x_stride; A.ab_stride = ab_stride;
    if (ckpt) set_ckpt(A, ckpt);
    A.states = const_cast<float*>(states);
    A.dh = dh; A.dh_stride = dh_stride; A.d_state = d_state;
    A.dx = dx; A.dx_stride = dx_stride; A.da = da; A.db = db; A.dab_stride = dab_stride;
    A.d_a_log = d_a_log; A.d_dt_bias = d_dt_bias; A.d_state0 = d_state0;
    auto on16 = [&](const void* p, int64_t stride) { return stride * elem_size(dt) % 16 == 0 && aligned(p, 16); };
    A.vec8 = C % 8 == 0 && on16(dh, dh_stride) &&
             (ckpt || (on16(x, x_stride) && on16(a, ab_stride) && on16(b, ab_stride)));
    return from_hip(gdnt::launch_scan_backward(A, (hipStream_t)stream));
}

GDN_EXPORT int32_t gdnt_conv_backward(const gdn_dims* dims, const void* conv_w, const void* x, int64_t x_stride,
                                      const void* dy, int32_t dy_dtype, int64_t dy_stride, const gdn_batch* batch,
                                      gdn_conv_pool conv, int32_t activation, const float* d_window, void* dx,
                                      int64_t dx_stride, float* d_conv_w, float* d_window0, void* workspace,
                                      size_t ws_bytes, int32_t* err, void* stream) {
    int32_t st;
    if ((st = gdn::dims_status(dims)) != GDN_OK) return st;
    if ((st = check_batch(batch)) != GDN_OK) return st;
    if (!conv_w || !d_conv_w || !dtype_ok(dy_dtype) || (activation != 0 && activation != 1)) return GDN_ERR_ARG;
    const int64_t C = 2 * (int64_t)dims->h_k * dims->d_k + (int64_t)dims->h_v * dims->d_v;
    const int32_t dt = dims->act_dtype;
    if ((st = check_conv_size(batch->n_rows, C)) != GDN_OK) return st;
    gdn_batch bt = *batch;
    if (bt.n_seqs == 0) bt.n_rows = 0;
    if (conv.base && bt.n_seqs > 0 &&
        (conv.rows < dims->conv_w - 1 || conv.n_pages < 0 || conv.page_stride < (int64_t)conv.rows * C))
        return GDN_ERR_ARG;
    if (!aligned(conv.base, (size_t)elem_size(dt)) || !aligned(conv_w, (size_t)elem_size(dt))) return GDN_ERR_ARG;
    if (bt.n_rows > 0) {
        if (!rows_ok(x, x_stride, C, dt) || !rows_ok(dy, dy_stride, C, dy_dtype) || !rows_ok(dx, dx_stride, C, dt))
            return GDN_ERR_ARG;
        if (!workspace || !aligned(workspace, 256)) return GDN_ERR_ARG;
    }
    if (ws_bytes < conv_ws(bt.n_rows, C, gdnt::conv_tiles(bt.n_rows, C))) return GDN_ERR_ARG;
    gdnt::ConvBwdArgs A{};
    A.x = x; A.x_stride = x_stride; A.dy = dy; A.dy_stride = dy_stride; A.n_rows = bt.n_rows;
    A.cu = bt.cu_seqlens; A.page_idx = bt.page_idx; A.has_init = bt.has_init; A.n_seqs = bt.n_seqs;
    A.max_len = bt.max_seqlen;
    A.conv_w = conv_w; A.window = conv.base; A.window_stride = conv.page_stride;
    A.page_limit = conv.base ? conv.n_pages : INT32_MAX;
    A.d_window = d_window; A.dx = dx; A.dx_stride = dx_stride; A.d_conv_w = d_conv_w; A.d_window0 = d_window0;
    A.map = static_cast<int32_t*>(workspace);
    A.part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      (size_t)n_tiles(bt.n_rows) * gdnt::kTileRows * sizeof(int32_t));
    A.C = (int32_t)C; A.activation = activation; A.act_dtype = dt; A.dy_dtype = dy_dtype; A.err = err;
    A.vec = C % 4 == 0 && rows_vec(x, x_stride, dt) && rows_vec(dy, dy_stride, dy_dtype) && rows_vec(dx, dx_stride, dt);
    return from_hip(gdnt::launch_conv_backward(A, (hipStream_t)stream));
}
