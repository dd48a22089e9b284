// gdnl_api.cpp -- the C ABI of include/gdn_linear.h: argument validation,
// workspace layout and kernel launches.  As in gdn_api.cpp every check runs on
// the host before anything is launched.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/gdn_linear.h"
#include "gdnl_kernels.h"

#define GDN_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

// Rows of a segment, at least, and workgroups (segments times value heads)
// from which on segments grow longer instead of more: two to a compute unit
// (512, 1024, 2048 take 467, 490, 545 us forward and 2175, 2320, 2605 with the
// backward pass over 4 x 8192 rows of 32 heads), and one where segments are short
// and states wide, whose reading and writing then counts (256 and 512 take 71 and
// 80 us over 2000 rows of 32 heads of 128 x 128, 93 and 100 us over 4000).
constexpr int32_t kSegMin = 128, kSegShort = 512;
constexpr int64_t kSegGroups = 512;
// Batches whose longest sequence has at most kSegNone rows are not cut, the states
// between segments costing two more launches and another reading of k and v; where
// sequences times heads are fewer than kSegFew, batches of at most kSegFewNone
// (900 rows of 8 heads 93 us uncut and 40 cut, 4 x 1000 rows of 32 heads 107 and
// 139), and fewer than twice as many for fp32 rows, whose chunks take longer (4 x
// 1000 rows of 32 heads 240 uncut and 205 cut, 8 prompts of up to 656 167 and 189).
constexpr int32_t kSegNone = 1024, kSegFewNone = 256;
constexpr int64_t kSegFew = 128;
// A backward pass takes no longer ones: the gradients of the decays are sums over
// the rows to a segment's ends, whose rounding grows with them.
constexpr int64_t kSegBack = 2048;
constexpr int32_t kSegWhole = INT32_MAX;  // every sequence is one segment
constexpr int64_t kMaxGroups = (1 << 23) - 1;  // of 512 threads: HIP launches fewer than 2^32 threads

int64_t elem_size(int32_t dt) { return dt == GDN_BF16 ? 2 : 4; }
bool dtype_ok(int32_t dt) { return dt == GDN_F32 || dt == GDN_BF16; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int32_t from_hip(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }
size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

bool rows_ok(const void* p, int64_t stride, int64_t width, int32_t dt) {
    // a chunk's rows are addressed by 32-bit byte offsets
    return p && stride >= width && stride <= (1 << 24) && aligned(p, (size_t)elem_size(dt));
}
// `bytes`: what rows and heads have to be multiples of.
bool rows_on(const void* p, int64_t stride, int64_t d, int32_t dt, int64_t bytes) {
    return stride * elem_size(dt) % bytes == 0 && d * elem_size(dt) % bytes == 0 && aligned(p, (size_t)bytes);
}

int32_t check_state_dims(const gdnl_dims* d) {
    if (!d || d->h_v <= 0 || d->d_k <= 0 || d->d_v <= 0 || !dtype_ok(d->state_dtype)) return GDN_ERR_ARG;
    if ((int64_t)d->h_v * d->d_v > (1 << 24) || (int64_t)d->h_v * d->d_k > (1 << 24)) return GDN_ERR_ARG;
    if ((int64_t)d->h_v * d->d_k * d->d_v > ((int64_t)1 << 31)) return GDN_ERR_ARG;
    return GDN_OK;
}
int32_t check_dims(const gdnl_dims* d) {
    const int32_t st = check_state_dims(d);
    if (st != GDN_OK) return st;
    if (d->h_k <= 0 || d->h_v % d->h_k != 0 || !dtype_ok(d->act_dtype) || !std::isfinite(d->scale)) return GDN_ERR_ARG;
    return d->d_k > gdnl::kMaxDim || d->d_v > gdnl::kMaxDim ? GDN_ERR_UNSUPPORTED : GDN_OK;
}
int32_t check_rows(int64_t n_rows) { return n_rows >= 0 && n_rows <= INT32_MAX - 1024 ? GDN_OK : GDN_ERR_ARG; }
int32_t check_batch(const gdn_batch* b) {
    if (!b || b->n_seqs < 0 || b->max_seqlen < 0 || check_rows(b->n_rows) != GDN_OK) return GDN_ERR_ARG;
    if (b->n_seqs > (1 << 28)) return GDN_ERR_ARG;
    if (b->n_seqs > 0 && (!b->cu_seqlens || !b->page_idx)) return GDN_ERR_ARG;
    return GDN_OK;
}
int32_t check_pool(const gdnl_dims* d, const gdn_state_pool& s) {
    // a segment's word holds 4 * page + 2 bits
    if (!s.base || s.n_pages < 0 || s.n_pages > (1 << 29) - 1) return GDN_ERR_ARG;
    if (s.page_stride < (int64_t)d->h_v * d->d_k * d->d_v) return GDN_ERR_ARG;
    return aligned(s.base, (size_t)elem_size(d->state_dtype)) ? GDN_OK : GDN_ERR_ARG;
}

// Rows of a segment for a batch of n_rows: as few as leave about kSegGroups
// workgroups.
int64_t seg_rows(int64_t n_rows, const gdnl_dims* d, bool backward) {
    const int64_t most_short = d->d_k > 64 || d->d_v > 64 ? kSegGroups / 2 : kSegGroups;
    int64_t len = kSegMin;
    while (len < n_rows && (n_rows + len - 1) / len * d->h_v > (len < kSegShort ? most_short : kSegGroups) &&
           !(backward && len == kSegBack))
        len *= 2;
    return len;
}
int64_t slots_of(int64_t n_seqs, int64_t n_rows, int64_t len) { return n_seqs + (n_rows + len - 1) / len + 1; }
// The most borders between segments that a batch of up to n_rows rows has, and slots.
int64_t most_borders(int64_t n_rows, int64_t heads, bool backward) {
    const int64_t by_rows = (n_rows + kSegMin - 1) / kSegMin, by_groups = kSegGroups / heads;
    int64_t most = by_rows < by_groups ? by_rows : by_groups;
    if (backward && most < (n_rows + kSegBack - 1) / kSegBack) most = (n_rows + kSegBack - 1) / kSegBack;
    return most < 1 ? 1 : most;
}
int64_t most_slots(int64_t n_seqs, int64_t borders) { return n_seqs + borders + 1; }

// The chunked kernels' grid, rounded up to whole key heads on every XCD, is beyond a launch.
bool too_many(int64_t slots, const gdnl_dims* d) {
    return slots * d->h_v + 7 * (int64_t)(d->h_v / d->h_k) > kMaxGroups;
}

struct Ws {
    size_t segs, seqs, total, gates, before, copy, after, rows, cols, last, first, ends, gate, part, all;
};
// asked: GDNL_ASKS_* of a backward call, 0 of a forward one.
Ws layout(const gdnl_dims* d, int64_t slots, int64_t borders, int64_t n_seqs, int64_t n_rows, bool backward, int32_t asked) {
    Ws w{};
    const size_t H = (size_t)d->h_v, size = (size_t)d->d_k * d->d_v;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at = round_up(at + bytes);
        return here;
    };
    w.segs = take((size_t)slots * sizeof(gdnl::SegWord));
    w.seqs = take((size_t)n_seqs * sizeof(gdnl::SeqSlots));
    w.total = take((size_t)slots * H * sizeof(double));
    w.gates = take(H * (size_t)n_rows * sizeof(float4));
    w.before = take((size_t)borders * H * size * sizeof(float));
    if (!backward) w.copy = take((size_t)borders * H * size * sizeof(float));
    if (backward) {
        w.after = take((size_t)borders * H * size * sizeof(float));
        w.rows = take(H * (size_t)n_rows * sizeof(float));
        w.cols = take(H * (size_t)n_rows * sizeof(float));
        // a state for every sequence only where the decays' gradient reads what is not an argument
        const size_t whole = (size_t)n_seqs * H * size * sizeof(float);
        w.last = take((asked & GDNL_ASKS_DG) && (asked & GDNL_ASKS_D_STATE) ? whole : 0);
        w.first = take((asked & GDNL_ASKS_DG) && !(asked & GDNL_ASKS_D_STATE0) ? whole : 0);
        w.ends = take((size_t)(slots + n_seqs) * H * sizeof(double));
        w.gate = take((size_t)slots * H * sizeof(double));
        if (d->h_k != d->h_v) w.part = take((size_t)n_rows * H * (size_t)d->d_k * sizeof(float));
    }
    w.all = at;
    return w;
}

gdnl::States pages_of(const gdnl_dims* d, const gdn_state_pool& s) {
    return gdnl::States{s.base, gdnl::kByPage, d->state_dtype == GDN_BF16 ? 1 : 0, s.page_stride,
                        (int64_t)d->d_k * d->d_v, d->d_v, 1};
}
gdnl::States dense(const gdnl_dims* d, const float* p, int32_t at) {
    const int64_t size = (int64_t)d->d_k * d->d_v;
    return gdnl::States{const_cast<float*>(p), p ? at : (int32_t)gdnl::kNoState, 0, size * d->h_v, size, d->d_v, 1};
}
gdnl::States turned(gdnl::States s) {
    const int32_t rs = s.rs;
    s.rs = s.cs;
    s.cs = rs;
    return s;
}

struct Plan {
    int64_t len, slots, segments;  // rows of a segment; segments of the call and, at most, of a sequence
    int64_t borders;               // between segments of a sequence
    bool split;  // sequences may have several segments
};
Plan plan_of(const gdnl_dims* d, const gdn_batch* b, bool backward) {
    Plan p;
    p.len = seg_rows(b->n_rows, d, backward);
    const int64_t most = b->max_seqlen > 0 && b->max_seqlen < b->n_rows ? b->max_seqlen : b->n_rows;  // rows of a sequence
    const int64_t whole = (int64_t)b->n_seqs * d->h_v < (d->act_dtype == GDN_F32 ? 2 * kSegFew : kSegFew) ? kSegFewNone : kSegNone;
    p.split = most > p.len && most > whole;
    if (!p.split) p.len = kSegWhole;
    p.slots = slots_of(b->n_seqs, b->n_rows, p.len);
    p.segments = (most + p.len - 1) / p.len;
    p.borders = p.split ? (b->n_rows + p.len - 1) / p.len : 0;
    return p;
}

}  // namespace

GDN_EXPORT int32_t gdnl_attend_workspace_bytes(const gdnl_dims* dims, int32_t n_seqs, int64_t n_rows, int32_t backward,
                                               size_t* out_bytes) {
    int32_t st;
    if ((st = check_dims(dims)) != GDN_OK) return st;
    constexpr int32_t all = GDNL_ASKS | GDNL_ASKS_DG | GDNL_ASKS_D_STATE | GDNL_ASKS_D_STATE0;
    if (!out_bytes || n_seqs < 0 || n_seqs > (1 << 28)) return GDN_ERR_ARG;
    if (backward != 0 && backward != 1 && (!(backward & GDNL_ASKS) || (backward & ~all))) return GDN_ERR_ARG;
    if ((st = check_rows(n_rows)) != GDN_OK) return st;
    const int32_t asked = backward == 1 ? GDNL_ASKS_DG | GDNL_ASKS_D_STATE : backward;  // 1: the most
    const int64_t borders = most_borders(n_rows, dims->h_v, backward != 0), slots = most_slots(n_seqs, borders);
    if (too_many(slots, dims)) return GDN_ERR_ARG;
    *out_bytes = layout(dims, slots, borders, n_seqs, n_rows, backward != 0, asked).all;
    return GDN_OK;
}

GDN_EXPORT int32_t gdnl_attend_forward(const gdnl_dims* dims, const void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, const void* v, int64_t v_stride, const float* g,
                                       int64_t g_stride, const gdn_batch* batch, gdn_state_pool state_in,
                                       gdn_state_pool state_out, void* o, int64_t o_stride, void* workspace,
                                       size_t ws_bytes, int32_t* err, void* stream) {
    int32_t st;
    if ((st = check_dims(dims)) != GDN_OK) return st;
    if ((st = check_batch(batch)) != GDN_OK) return st;
    if (batch->n_seqs == 0) return GDN_OK;
    if ((st = check_pool(dims, state_in)) != GDN_OK || (st = check_pool(dims, state_out)) != GDN_OK) return st;
    const int32_t dt = dims->act_dtype, H = dims->h_v, per = H / dims->h_k;
    const int64_t wk = (int64_t)dims->h_k * dims->d_k, wv = (int64_t)H * dims->d_v;
    if (batch->n_rows > 0 && (!rows_ok(q, q_stride, wk, dt) || !rows_ok(k, k_stride, wk, dt) ||
                              !rows_ok(v, v_stride, wv, dt) || !rows_ok(o, o_stride, wv, dt) || !g || !aligned(g, 4) ||
                              (g_stride != 0 && (g_stride < H || g_stride > (1 << 24)))))
        return GDN_ERR_ARG;
    const hipStream_t s = (hipStream_t)stream;
    const int32_t limit = state_in.n_pages < state_out.n_pages ? state_in.n_pages : state_out.n_pages;
    if (batch->max_seqlen > 0 && batch->max_seqlen <= GDNL_TOKEN_ROWS) {
        if ((int64_t)batch->n_seqs * H > kMaxGroups) return GDN_ERR_ARG;
        gdnl::TokenArgs A{};
        A.cu = batch->cu_seqlens; A.page_idx = batch->page_idx; A.has_init = batch->has_init;
        A.n_seqs = batch->n_seqs; A.max_len = batch->max_seqlen; A.page_limit = limit; A.n_rows = batch->n_rows;
        A.q = q; A.k = k; A.v = v; A.g = g; A.o = o;
        A.q_stride = q_stride; A.k_stride = k_stride; A.v_stride = v_stride; A.g_stride = g_stride; A.o_stride = o_stride;
        A.st_in = state_in.base; A.st_in_stride = state_in.page_stride;
        A.st_out = state_out.base; A.st_out_stride = state_out.page_stride;
        A.heads = H; A.per = per; A.dk = dims->d_k; A.dv = dims->d_v; A.scale = dims->scale; A.err = err;
        A.act_bf16 = dt == GDN_BF16; A.state_bf16 = dims->state_dtype == GDN_BF16;
        const int64_t four = 4 * elem_size(dims->state_dtype);
        A.vec = rows_on(state_in.base, state_in.page_stride, dims->d_v, dims->state_dtype, four) &&
                rows_on(state_out.base, state_out.page_stride, dims->d_v, dims->state_dtype, four);
        return from_hip(gdnl::launch_tokens(A, s));
    }
    const Plan p = plan_of(dims, batch, false);
    if (too_many(p.slots, dims)) return GDN_ERR_ARG;
    const Ws w = layout(dims, p.slots, p.borders, batch->n_seqs, batch->n_rows, false, 0);
    if (!workspace || !aligned(workspace, 256) || ws_bytes < w.all) return GDN_ERR_ARG;
    char* const ws = static_cast<char*>(workspace);
    gdnl::SegmentArgs G{};
    G.cu = batch->cu_seqlens; G.page_idx = batch->page_idx; G.n_seqs = batch->n_seqs; G.n_rows = batch->n_rows;
    G.n_slots = p.slots; G.len = (int32_t)p.len; G.max_len = batch->max_seqlen; G.page_limit = limit;
    G.segs = reinterpret_cast<gdnl::SegWord*>(ws + w.segs);
    G.seqs = reinterpret_cast<gdnl::SeqSlots*>(ws + w.seqs);
    G.err = err;
    if (batch->n_rows == 0) return from_hip(gdnl::launch_segments(G, s));
    float* const before = reinterpret_cast<float*>(ws + w.before);
    double* const total = reinterpret_cast<double*>(ws + w.total);

    gdnl::AttendArgs A{};
    A.segs = G.segs; A.n_slots = p.slots; A.n_rows = batch->n_rows;
    A.q = {q, q_stride, per};
    A.k = {k, k_stride, per};
    A.v = {v, v_stride, 1};
    A.vec = rows_on(q, q_stride, dims->d_k, dt, 16) && rows_on(k, k_stride, dims->d_k, dt, 16) &&
            rows_on(v, v_stride, dims->d_v, dt, 16) && rows_on(o, o_stride, dims->d_v, dt, 16);
    A.has_init = batch->has_init; A.len = (int32_t)p.len;
    A.dk = dims->d_k; A.dv = dims->d_v; A.heads = H; A.per = per;
    A.f_p = A.f_i = dims->scale; A.f_u = 1.0f;
    A.gates = reinterpret_cast<const float4*>(ws + w.gates);
    gdnl::DecayArgs D{G.segs, p.slots, batch->n_rows, H, g, g_stride, reinterpret_cast<float4*>(ws + w.gates), total};
    hipError_t e = gdnl::launch_segments_decays(G, D, s);
    if (e != hipSuccess) return from_hip(e);
    if (p.split) {
        A.out = A.mid = dense(dims, before, gdnl::kByBorder);
        if ((e = gdnl::launch_attend(A, gdnl::kLocal, false, dt == GDN_BF16, s)) != hipSuccess) return from_hip(e);
        float* const copy = reinterpret_cast<float*>(ws + w.copy);
        gdnl::ScanArgs C{G.seqs, batch->page_idx, batch->has_init, batch->n_seqs, H, dims->d_k * dims->d_v, 0,
                         pages_of(dims, state_in), before, total, copy};
        A.copy = dense(dims, copy, gdnl::kByBorder);
        if ((e = gdnl::launch_state_scan(C, p.segments, s)) != hipSuccess) return from_hip(e);
    }
    A.in = pages_of(dims, state_in);
    A.out = pages_of(dims, state_out);
    A.o = o; A.o_stride = o_stride;
    A.o_f32 = dt == GDN_F32;
    return from_hip(gdnl::launch_attend(A, gdnl::kAttend, false, dt == GDN_BF16, s));
}

GDN_EXPORT int32_t gdnl_attend_backward(const gdnl_dims* dims, const void* q, int64_t q_stride, const void* k,
                                        int64_t k_stride, const void* v, int64_t v_stride, const float* g,
                                        int64_t g_stride, const gdn_batch* batch, gdn_state_pool state_in,
                                        const void* d_o, int64_t do_stride, const float* d_state, void* dq,
                                        int64_t dq_stride, void* dk, int64_t dk_stride, void* dv, int64_t dv_stride,
                                        float* dg, float* d_state0, void* workspace, size_t ws_bytes, int32_t* err,
                                        void* stream) {
    int32_t st;
    if ((st = check_dims(dims)) != GDN_OK) return st;
    if ((st = check_batch(batch)) != GDN_OK) return st;
    const int32_t dt = dims->act_dtype, H = dims->h_v, per = H / dims->h_k;
    const hipStream_t s = (hipStream_t)stream;
    if (!aligned(dg, 4) || !aligned(d_state, 4) || !aligned(d_state0, 4)) return GDN_ERR_ARG;
    if (g_stride != 0 && (g_stride < H || g_stride > (1 << 24))) return GDN_ERR_ARG;
    const bool one_decay = g_stride == 0;
    if (batch->n_seqs == 0) return dg && one_decay ? from_hip(gdnl::launch_gate_sum(nullptr, 0, H, dg, s)) : GDN_OK;
    if ((st = check_pool(dims, state_in)) != GDN_OK) return st;
    const int64_t wk = (int64_t)dims->h_k * dims->d_k, wv = (int64_t)H * dims->d_v;
    if (batch->n_rows > 0 &&
        (!rows_ok(q, q_stride, wk, dt) || !rows_ok(k, k_stride, wk, dt) || !rows_ok(v, v_stride, wv, dt) ||
         !rows_ok(d_o, do_stride, wv, dt) || !rows_ok(dq, dq_stride, wk, dt) || !rows_ok(dk, dk_stride, wk, dt) ||
         !rows_ok(dv, dv_stride, wv, dt) || !g || !aligned(g, 4)))
        return GDN_ERR_ARG;
    const Plan p = plan_of(dims, batch, true);
    if (too_many(p.slots, dims)) return GDN_ERR_ARG;
    const int32_t asked = (dg ? GDNL_ASKS_DG : 0) | (d_state ? GDNL_ASKS_D_STATE : 0) | (d_state0 ? GDNL_ASKS_D_STATE0 : 0);
    const Ws w = layout(dims, p.slots, p.borders, batch->n_seqs, batch->n_rows, true, asked);
    if (!workspace || !aligned(workspace, 256) || ws_bytes < w.all) return GDN_ERR_ARG;
    char* const ws = static_cast<char*>(workspace);
    const int32_t size = dims->d_k * dims->d_v;
    gdnl::SegmentArgs G{};
    G.cu = batch->cu_seqlens; G.page_idx = batch->page_idx; G.n_seqs = batch->n_seqs; G.n_rows = batch->n_rows;
    G.n_slots = p.slots; G.len = (int32_t)p.len; G.max_len = batch->max_seqlen; G.page_limit = state_in.n_pages;
    G.segs = reinterpret_cast<gdnl::SegWord*>(ws + w.segs);
    G.seqs = reinterpret_cast<gdnl::SeqSlots*>(ws + w.seqs);
    G.pass_src = d_state; G.pass_dst = d_state0; G.pass_width = (int64_t)H * size;
    G.err = err;
    hipError_t e = hipSuccess;
    if (batch->n_rows == 0) {
        e = gdnl::launch_segments(G, s);
        return e == hipSuccess && dg && one_decay ? from_hip(gdnl::launch_gate_sum(nullptr, 0, H, dg, s)) : from_hip(e);
    }
    float* const before = reinterpret_cast<float*>(ws + w.before);
    float* const after = reinterpret_cast<float*>(ws + w.after);
    float* const rows = reinterpret_cast<float*>(ws + w.rows);
    float* const cols = reinterpret_cast<float*>(ws + w.cols);
    float* const last = reinterpret_cast<float*>(ws + w.last);
    float* const part = reinterpret_cast<float*>(ws + w.part);
    double* const total = reinterpret_cast<double*>(ws + w.total);

    const gdnl::Rows rq{q, q_stride, per}, rk{k, k_stride, per}, rv{v, v_stride, 1}, ro{d_o, do_stride, 1};
    gdnl::AttendArgs A{};
    A.vec = rows_on(q, q_stride, dims->d_k, dt, 16) && rows_on(k, k_stride, dims->d_k, dt, 16) &&
            rows_on(v, v_stride, dims->d_v, dt, 16) && rows_on(d_o, do_stride, dims->d_v, dt, 16) &&
            rows_on(dq, dq_stride, dims->d_k, dt, 16) && rows_on(dk, dk_stride, dims->d_k, dt, 16) &&
            rows_on(dv, dv_stride, dims->d_v, dt, 16);
    A.segs = G.segs; A.n_slots = p.slots; A.n_rows = batch->n_rows;
    A.has_init = batch->has_init; A.heads = H; A.per = per; A.len = (int32_t)p.len;
    A.gates = reinterpret_cast<const float4*>(ws + w.gates);
    gdnl::DecayArgs D{G.segs, p.slots, batch->n_rows, H, g, g_stride, reinterpret_cast<float4*>(ws + w.gates), total};
    if ((e = gdnl::launch_segments_decays(G, D, s)) != hipSuccess) return from_hip(e);
    const gdnl::States ends = dense(dims, d_state, gdnl::kBySeq);
    const gdnl::States at_borders = dense(dims, before, gdnl::kByBorder), grad_borders = dense(dims, after, gdnl::kByBorder);
    if (p.split) {
        // S at every border, then its gradient there
        A.k = rk; A.v = rv; A.dk = dims->d_k; A.dv = dims->d_v; A.f_u = 1.0f;
        A.out = at_borders;
        if ((e = gdnl::launch_attend(A, gdnl::kLocal, false, dt == GDN_BF16, s)) != hipSuccess) return from_hip(e);
        gdnl::ScanArgs C{G.seqs, batch->page_idx, batch->has_init, batch->n_seqs, H, size, 0, pages_of(dims, state_in),
                         before, total, nullptr};
        if ((e = gdnl::launch_state_scan(C, p.segments, s)) != hipSuccess) return from_hip(e);
        A.k = rq; A.v = ro; A.f_u = dims->scale;
        A.out = grad_borders;
        if ((e = gdnl::launch_attend(A, gdnl::kLocal, true, dt == GDN_BF16, s)) != hipSuccess) return from_hip(e);
        C.in = ends; C.back = 1; C.local = after;
        if ((e = gdnl::launch_state_scan(C, p.segments, s)) != hipSuccess) return from_hip(e);
    }
    const bool grouped = per > 1;
    auto group = [&](void* out, int64_t stride) {
        const int64_t most = batch->max_seqlen > 0 && batch->max_seqlen < p.len ? batch->max_seqlen
                             : p.len < batch->n_rows                            ? p.len
                                                                                : batch->n_rows;
        gdnl::GroupArgs B{G.segs, p.slots, H, per, dims->d_k, dt == GDN_BF16,
                          rows_on(out, stride, dims->d_k, dt, 4 * elem_size(dt)), most, part, out, stride};
        return grouped ? gdnl::launch_group_sum(B, s) : hipSuccess;
    };
    auto to_keys = [&](void* out, int64_t stride) {
        A.o = grouped ? static_cast<void*>(part) : out;
        A.o_stride = grouped ? (int64_t)H * dims->d_k : stride;
        A.o_f32 = grouped || dt == GDN_F32;
    };
    // dq: linear attention of d_o over the rows of v and k
    A.q = ro; A.k = rv; A.v = rk; A.x = rq;
    A.dk = dims->d_v; A.dv = dims->d_k;
    A.f_p = A.f_i = dims->scale; A.f_u = 1.0f;
    A.in = turned(pages_of(dims, state_in));
    A.mid = turned(at_borders);
    A.out = turned(dense(dims, dg && d_state ? last : nullptr, gdnl::kBySeq));
    A.dot = rows;
    to_keys(dq, dq_stride);
    if ((e = gdnl::launch_attend(A, dg ? gdnl::kDotRows : gdnl::kAttend, false, dt == GDN_BF16, s)) != hipSuccess) return from_hip(e);
    if ((e = group(dq, dq_stride)) != hipSuccess) return from_hip(e);
    // dk: of v over d_o and q, backward in time
    A.q = rv; A.k = ro; A.v = rq; A.x = rk;
    A.f_i = 1.0f; A.f_u = dims->scale;
    A.in = turned(ends);
    A.mid = turned(grad_borders);
    A.out = gdnl::States{};
    A.dot = cols;
    to_keys(dk, dk_stride);
    if ((e = gdnl::launch_attend(A, dg ? gdnl::kDot : gdnl::kAttend, true, dt == GDN_BF16, s)) != hipSuccess) return from_hip(e);
    if ((e = group(dk, dk_stride)) != hipSuccess) return from_hip(e);
    // dv: of k over q and d_o, backward in time, and the initial state's gradient
    A.q = rk; A.k = rq; A.v = ro;
    A.dk = dims->d_k; A.dv = dims->d_v;
    A.in = ends;
    A.mid = grad_borders;
    float* const first = dg && !d_state0 ? reinterpret_cast<float*>(ws + w.first) : d_state0;
    A.out = dense(dims, first, gdnl::kBySeq);
    A.zero_uninit = 1;
    A.o = dv; A.o_stride = dv_stride; A.o_f32 = dt == GDN_F32;
    if ((e = gdnl::launch_attend(A, gdnl::kAttend, true, dt == GDN_BF16, s)) != hipSuccess) return from_hip(e);
    if (!dg) return GDN_OK;
    gdnl::GateArgs T{G.segs, p.slots, batch->n_rows, H, size, (int32_t)p.len, g, g_stride, rows, cols, before, after, last, d_state,
                     G.seqs, batch->page_idx, batch->has_init, batch->n_seqs, pages_of(dims, state_in), first,
                     reinterpret_cast<double*>(ws + w.ends), dg, one_decay ? reinterpret_cast<double*>(ws + w.gate) : nullptr};
    if ((e = gdnl::launch_gate(T, s)) != hipSuccess || !one_decay) return from_hip(e);
    return from_hip(gdnl::launch_gate_sum(T.part, p.slots, H, dg, s));
}

// ------------------------------------------------------------- rotation

namespace {

int32_t check_rotate(const gdnl_rotate_dims* d) {
    if (!d || d->h_q < 0 || d->h_k < 0 || (int64_t)d->h_q + d->h_k > (1 << 16)) return GDN_ERR_ARG;
    if (d->d <= 0 || d->d % 2 != 0 || d->rot < 0 || d->rot > d->d || d->rot % 2 != 0) return GDN_ERR_ARG;
    if (!dtype_ok(d->act_dtype) || !std::isfinite(d->eps) || d->eps < 0.0f) return GDN_ERR_ARG;
    if ((d->norm != GDNL_NORM_RMS && d->norm != GDNL_NORM_L2) ||
        (d->pairs != GDNL_PAIRS_HALVES && d->pairs != GDNL_PAIRS_NEIGHBOURS))
        return GDN_ERR_ARG;
    return d->d > 256 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

bool fours(const gdnl_rotate_dims* d, int32_t heads, const void* p, int64_t stride) {
    return heads == 0 || rows_on(p, stride, d->d, d->act_dtype, 4 * elem_size(d->act_dtype));
}

gdnl::RotateArgs rotate_args(const gdnl_rotate_dims* d, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const float* wq, const float* wk, const int32_t* pos,
                             const float* inv_freq, int64_t n_rows) {
    gdnl::RotateArgs A{};
    A.x[0] = q; A.x[1] = k; A.x_stride[0] = q_stride; A.x_stride[1] = k_stride;
    A.w[0] = wq; A.w[1] = wk; A.pos = pos; A.inv_freq = inv_freq; A.n_rows = n_rows;
    A.heads[0] = d->h_q; A.heads[1] = d->h_k; A.d = d->d; A.rot = d->rot;
    A.neighbours = d->pairs == GDNL_PAIRS_NEIGHBOURS; A.bf16 = d->act_dtype == GDN_BF16;
    A.over = d->norm == GDNL_NORM_RMS ? (float)d->d : 1.0f; A.eps = d->eps;
    // four pairs side by side are all halves or all neighbours
    A.vec = d->d % 8 == 0 && (d->pairs == GDNL_PAIRS_NEIGHBOURS || d->rot % 8 == 0) && fours(d, d->h_q, q, q_stride) &&
            fours(d, d->h_k, k, k_stride);
    return A;
}

int32_t check_rotate_rows(const gdnl_rotate_dims* d, const void* q, int64_t q_stride, const void* k, int64_t k_stride) {
    const int32_t dt = d->act_dtype;
    if (d->h_q > 0 && !rows_ok(q, q_stride, (int64_t)d->h_q * d->d, dt)) return GDN_ERR_ARG;
    if (d->h_k > 0 && !rows_ok(k, k_stride, (int64_t)d->h_k * d->d, dt)) return GDN_ERR_ARG;
    return GDN_OK;
}

}  // namespace

GDN_EXPORT int32_t gdnl_rotate_workspace_bytes(const gdnl_rotate_dims* dims, int64_t n_rows, size_t* out_bytes) {
    const int32_t st = check_rotate(dims);
    if (st != GDN_OK) return st;
    if (!out_bytes || check_rows(n_rows) != GDN_OK) return GDN_ERR_ARG;
    *out_bytes = round_up((size_t)gdnl::rotate_groups(n_rows) * 2 * (size_t)dims->d * sizeof(double));
    return GDN_OK;
}

GDN_EXPORT int32_t gdnl_rotate_forward(const gdnl_rotate_dims* dims, const void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, const float* wq, const float* wk, const int32_t* pos,
                                       const float* inv_freq, int64_t n_rows, void* yq, int64_t yq_stride, void* yk,
                                       int64_t yk_stride, void* stream) {
    int32_t st;
    if ((st = check_rotate(dims)) != GDN_OK) return st;
    if (check_rows(n_rows) != GDN_OK || !aligned(wq, 4) || !aligned(wk, 4)) return GDN_ERR_ARG;
    if (n_rows == 0 || dims->h_q + dims->h_k == 0) return GDN_OK;
    if (dims->rot > 0 && (!pos || !inv_freq || !aligned(pos, 4) || !aligned(inv_freq, 4))) return GDN_ERR_ARG;
    if ((st = check_rotate_rows(dims, q, q_stride, k, k_stride)) != GDN_OK) return st;
    if ((st = check_rotate_rows(dims, yq, yq_stride, yk, yk_stride)) != GDN_OK) return st;
    if ((dims->h_q > 0 && q == yq && q_stride != yq_stride) || (dims->h_k > 0 && k == yk && k_stride != yk_stride))
        return GDN_ERR_ARG;
    gdnl::RotateArgs A = rotate_args(dims, q, q_stride, k, k_stride, wq, wk, pos, inv_freq, n_rows);
    A.y[0] = yq; A.y[1] = yk; A.y_stride[0] = yq_stride; A.y_stride[1] = yk_stride;
    A.vec = A.vec && fours(dims, dims->h_q, yq, yq_stride) && fours(dims, dims->h_k, yk, yk_stride);
    return from_hip(gdnl::launch_rotate(A, false, (hipStream_t)stream));
}

GDN_EXPORT int32_t gdnl_rotate_backward(const gdnl_rotate_dims* dims, const void* q, int64_t q_stride, const void* k,
                                        int64_t k_stride, const float* wq, const float* wk, const int32_t* pos,
                                        const float* inv_freq, int64_t n_rows, const void* d_yq, int64_t d_yq_stride,
                                        const void* d_yk, int64_t d_yk_stride, void* dq, int64_t dq_stride, void* dk,
                                        int64_t dk_stride, float* dwq, float* dwk, void* workspace, size_t ws_bytes,
                                        void* stream) {
    int32_t st;
    if ((st = check_rotate(dims)) != GDN_OK) return st;
    if (check_rows(n_rows) != GDN_OK || !aligned(wq, 4) || !aligned(wk, 4) || !aligned(dwq, 4) || !aligned(dwk, 4))
        return GDN_ERR_ARG;
    const bool sums = dwq || dwk;
    if (n_rows > 0 && dims->h_q + dims->h_k > 0) {
        if (dims->rot > 0 && (!pos || !inv_freq || !aligned(pos, 4) || !aligned(inv_freq, 4))) return GDN_ERR_ARG;
        if ((st = check_rotate_rows(dims, q, q_stride, k, k_stride)) != GDN_OK) return st;
        if ((st = check_rotate_rows(dims, d_yq, d_yq_stride, d_yk, d_yk_stride)) != GDN_OK) return st;
        if ((st = check_rotate_rows(dims, dq, dq_stride, dk, dk_stride)) != GDN_OK) return st;
        if ((dims->h_q > 0 && d_yq == dq && d_yq_stride != dq_stride) ||
            (dims->h_k > 0 && d_yk == dk && d_yk_stride != dk_stride))
            return GDN_ERR_ARG;
    } else {
        n_rows = 0;
        if (!sums) return GDN_OK;
    }
    const size_t need = round_up((size_t)gdnl::rotate_groups(n_rows) * 2 * (size_t)dims->d * sizeof(double));
    if (sums && n_rows > 0 && (!workspace || !aligned(workspace, 256) || ws_bytes < need)) return GDN_ERR_ARG;
    gdnl::RotateArgs A = rotate_args(dims, q, q_stride, k, k_stride, wq, wk, pos, inv_freq, n_rows);
    A.dy[0] = d_yq; A.dy[1] = d_yk; A.dy_stride[0] = d_yq_stride; A.dy_stride[1] = d_yk_stride;
    A.y[0] = dq; A.y[1] = dk; A.y_stride[0] = dq_stride; A.y_stride[1] = dk_stride;
    A.vec = A.vec && fours(dims, dims->h_q, d_yq, d_yq_stride) && fours(dims, dims->h_k, d_yk, d_yk_stride) &&
            fours(dims, dims->h_q, dq, dq_stride) && fours(dims, dims->h_k, dk, dk_stride);
    A.dw[0] = dwq; A.dw[1] = dwk;
    A.part = sums ? static_cast<double*>(workspace) : nullptr;
    return from_hip(gdnl::launch_rotate(A, true, (hipStream_t)stream));
}

// ---------------------------------------------------------------- cache

namespace {

int32_t cache_call(const gdnl_dims* dims, int32_t n, const int32_t* page_idx, const int32_t* entry,
                   const gdn_state_pool& state, const gdnl_cache* cache, int32_t* err, void* stream, bool store) {
    int32_t st;
    if ((st = check_state_dims(dims)) != GDN_OK) return st;
    if (n < 0 || !cache || cache->n_entries < 0) return GDN_ERR_ARG;
    if (n == 0) return GDN_OK;
    if (!page_idx || !entry || !cache->q || !aligned(cache->q, 4) || !cache->scale || !aligned(cache->scale, 4))
        return GDN_ERR_ARG;
    if ((st = check_pool(dims, state)) != GDN_OK) return st;
    gdnl::CacheArgs A{};
    A.n = n; A.page = page_idx; A.entry = entry;
    A.st = state.base; A.st_stride = state.page_stride; A.n_pages = state.n_pages;
    A.bf16 = dims->state_dtype == GDN_BF16;
    A.q = cache->q; A.scale = cache->scale; A.n_entries = cache->n_entries;
    A.rows = (int64_t)dims->h_v * dims->d_k; A.dv = dims->d_v; A.err = err;
    A.vec = rows_on(state.base, state.page_stride, dims->d_v, dims->state_dtype, 4 * elem_size(dims->state_dtype));
    if (A.rows * ((A.dv + 63) / 64) / 64 + 1 > kMaxGroups / n) return GDN_ERR_ARG;
    return from_hip(gdnl::launch_cache(A, store, (hipStream_t)stream));
}

}  // namespace

GDN_EXPORT int32_t gdnl_cache_bytes(const gdnl_dims* dims, int32_t n_entries, size_t* q_bytes, size_t* scale_bytes) {
    const int32_t st = check_state_dims(dims);
    if (st != GDN_OK) return st;
    if (n_entries < 0) return GDN_ERR_ARG;
    const size_t rows = (size_t)n_entries * (size_t)dims->h_v * (size_t)dims->d_k;
    if (q_bytes) *q_bytes = rows * (size_t)dims->d_v;
    if (scale_bytes) *scale_bytes = rows * (size_t)((dims->d_v + 63) / 64) * sizeof(float);
    return GDN_OK;
}

GDN_EXPORT int32_t gdnl_cache_store(const gdnl_dims* dims, int32_t n, const int32_t* page_idx, const int32_t* entry,
                                    gdn_state_pool state, const gdnl_cache* cache, int32_t* err, void* stream) {
    return cache_call(dims, n, page_idx, entry, state, cache, err, stream, true);
}

GDN_EXPORT int32_t gdnl_cache_load(const gdnl_dims* dims, int32_t n, const int32_t* entry, const int32_t* page_idx,
                                   const gdnl_cache* cache, gdn_state_pool state, int32_t* err, void* stream) {
    return cache_call(dims, n, page_idx, entry, state, cache, err, stream, false);
}
