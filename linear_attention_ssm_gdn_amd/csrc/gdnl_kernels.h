// gdnl_kernels.h -- argument blocks and launchers of the operators of
// include/gdn_linear.h (the C ABI in gdnl_api.cpp validates arguments and
// calls these).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdnl {

constexpr int kChunk = 64;       // rows that meet each other by matrix products
constexpr int kThreads = 256;    // of every kernel here
constexpr int kMaxDim = 128;     // head dims of the attend kernels

// A run of one sequence's rows that a workgroup walks: packed rows
// [row, row + rows), rows 0 for a slot that no segment has.
struct Segment {
    int32_t seq, row, rows, page;
    bool first, last;            // of its sequence
};
struct SegWord { int32_t seq, row, rows, page; };  // page: page * 4 + 2 * last + first
// Where a sequence's segments stand: slots [slot, slot + n), n 0 for none.
struct SeqSlots { int32_t slot, n; };

// Segments of `len` rows (a multiple of 64) of every valid sequence: segment i
// of sequence s has slot s + cu[s] / len + i.  Valid sequences do not overlap,
// so their slots do not either, and all are below n_seqs + ceil(n_rows / len).
// Where row r begins a sequence's second or later segment stands border r / len:
// rows of one sequence's borders are len from each other, and those of another
// more, its own first segment lying between.  There are ceil(n_rows / len) borders
// however many sequences a batch has, and only cut ones have states at them.  By
// the same division of their first rows cut sequences differ from each other too.
struct SegmentArgs {
    const int32_t* cu; const int32_t* page_idx; int32_t n_seqs;
    int64_t n_rows, n_slots;
    int32_t len, max_len, page_limit;
    SegWord* segs; SeqSlots* seqs;
    // a backward pass hands the gradient of empty sequences through and clears
    // that of skipped ones: `pass_width` values a sequence, NULL src: zeros
    const float* pass_src; float* pass_dst; int64_t pass_width;
    int32_t* err;
};
hipError_t launch_segments(const SegmentArgs& a, hipStream_t s);

struct Rows {                    // packed rows of heads
    const void* p; int64_t stride;
    int32_t per;                 // value heads to a head of these rows
};

// Where a segment's state comes from or goes to.
enum StateAt { kNoState = 0, kByPage, kBySeq, kByBorder };
struct States {
    void* p; int32_t at, bf16;
    int64_t unit, head;          // elements from page (sequence, border) to the next, from head to head
    int32_t rs, cs;              // from row to row and column to column of the matrix the kernel holds
};

// For every row and head, G the inclusive sum of g log2(e) within the row's
// chunk of its segment: {G, what G's float leaves of it, e^G, e^{G_C - G}},
// e^{G_C} at a chunk's last row, and for every segment the sum over its rows.
struct DecayArgs {
    const SegWord* segs; int64_t n_slots, n_rows;
    int32_t heads;
    const float* g; int64_t g_stride;
    float4* gates;               // [heads][n_rows]
    double* total;               // [slot][heads]
};
hipError_t launch_segments_decays(const SegmentArgs& s, const DecayArgs& a, hipStream_t stream);

// One pass of linear attention over segments, forward or backward in time.
// For output row x and source row y of a chunk, y <= x forward, y >= x backward:
//   out_x = f_p sum_y e^{|G_x - G_y|}' (q_x . k_y) v_y + f_i e^{..} q_x^T S,
//   S <- e^{G_C} S + f_u sum_y e^{..} k_y v_y^T,
// forward with e^{G_x - G_y}, e^{G_x}, e^{G_C - G_y}, backward with e^{G_y -
// G_x}, e^{G_C - G_x}, e^{G_y}; G the inclusive sum of g within the chunk.
struct AttendArgs {
    const SegWord* segs; int64_t n_slots;
    Rows q, k, v, x;
    const float4* gates;         // of launch_segments_decays
    const uint8_t* has_init;
    int32_t dk, dv, heads, per;  // widths of q, k and of v, out; value heads, those to a key head
    float f_p, f_i, f_u;
    // in, out: at the ends of a sequence (out of local sums: at the border that the segment ends at);
    // mid: in of segments that begin at a border; copy: of the first segment of a cut sequence, whose page another
    // segment's workgroup may write (kNoState: no such page is written)
    States in, mid, copy, out;
    int32_t len;                 // rows of a segment
    int32_t zero_uninit;         // out is zero where has_init is 0
    void* o; int64_t o_stride; int32_t o_f32;
    int32_t vec;                 // all rows and heads on 16 bytes, those of o on four values
    float* dot;                  // [heads][n_rows]: see kDot, kDotRows
    int64_t n_rows;
};
enum AttendMode {
    kAttend = 0,
    kDot,        // also dot_x = x_x . (f_i part of out_x), over the columns
    kDotRows,    // the same, plus row sums less column sums of M_xy = (f_p e^{..} q_x.k_y)(x_x.v_y), y != x
    kLocal       // the state's sum over the segment alone, from zero
};
// mode kAttend, kDotRows or kLocal; back: kAttend, kDot or kLocal
hipError_t launch_attend_bf16(const AttendArgs& a, int mode, hipStream_t s);
hipError_t launch_attend_f32(const AttendArgs& a, int mode, hipStream_t s);
hipError_t launch_attend_bf16_back(const AttendArgs& a, int mode, hipStream_t s);
hipError_t launch_attend_f32_back(const AttendArgs& a, int mode, hipStream_t s);
inline hipError_t launch_attend(const AttendArgs& a, int mode, bool back, bool bf16, hipStream_t s) {
    if (back) return bf16 ? launch_attend_bf16_back(a, mode, s) : launch_attend_f32_back(a, mode, s);
    return bf16 ? launch_attend_bf16(a, mode, s) : launch_attend_f32(a, mode, s);
}

// At every border the state there in the place of the local sum of the segment
// in front of it (back: behind it).
struct ScanArgs {
    const SeqSlots* seqs; const int32_t* page_idx; const uint8_t* has_init;
    int32_t n_seqs, heads, size, back;   // size: dk * dv
    States in;
    float* local;                // [border][heads][size]
    const double* total;
    float* copy;                 // [first row / len][heads][size]: receives cut sequences' `in`, or NULL
};
hipError_t launch_state_scan(const ScanArgs& a, int64_t segments, hipStream_t s);  // of a sequence, at most

// dg_t = X + sum_{i >= t} (rows_i - cols_i) within a segment, X = <state, its
// gradient> at the segment's end.
struct GateArgs {
    const SegWord* segs; int64_t n_slots, n_rows;
    int32_t heads, size, len;
    const float* g; int64_t g_stride;
    const float* rows; const float* cols;          // [heads][n_rows]
    const float* before; const float* after;       // [border][heads][size]: the state and its gradient there
    const float* last; const float* d_state;       // [seq][heads][size]; d_state NULL: X is 0 at a sequence's end
    const SeqSlots* seqs; const int32_t* page_idx; const uint8_t* has_init;
    int32_t n_seqs; States start;                  // the pages, and
    const float* first;                            // [seq][heads][size]: their gradient
    double* ends;                                  // [slot, then seq][heads]
    float* dg;                                     // [n_rows][heads], or with g_stride 0:
    double* part;                                  // [slot][heads]
};
hipError_t launch_gate(const GateArgs& a, hipStream_t s);
hipError_t launch_gate_sum(const double* part, int64_t n_slots, int32_t heads, float* dg, hipStream_t s);

// out[row][h][c] = sum over a group's value heads of part[row][h * per + j][c], in order.
struct GroupArgs {
    const SegWord* segs; int64_t n_slots;
    int32_t heads, per, d, bf16, vec;   // vec: rows and heads on four values
    int64_t most_rows;                  // of a segment
    const float* part; void* out; int64_t stride;
};
hipError_t launch_group_sum(const GroupArgs& a, hipStream_t s);

// Sequences of a few rows, one workgroup to a sequence and value head.
struct TokenArgs {
    const int32_t* cu; const int32_t* page_idx; const uint8_t* has_init;
    int32_t n_seqs, max_len, page_limit; int64_t n_rows;
    const void* q; const void* k; const void* v; const float* g; void* o;
    int64_t q_stride, k_stride, v_stride, g_stride, o_stride;
    const void* st_in; int64_t st_in_stride; void* st_out; int64_t st_out_stride;
    int32_t heads, per, dk, dv, act_bf16, state_bf16, vec;
    float scale;
    int32_t* err;
};
hipError_t launch_tokens(const TokenArgs& a, hipStream_t s);

struct RotateArgs {
    const void* x[2]; const void* dy[2]; void* y[2];   // q, k; y: the output, or dx
    int64_t x_stride[2], dy_stride[2], y_stride[2];
    const float* w[2];
    const int32_t* pos; const float* inv_freq;
    int64_t n_rows;
    int32_t heads[2], d, rot, neighbours, bf16, vec;
    float over, eps;             // the sum of squares is divided by `over`
    double* part; float* dw[2];  // backward: [groups][2][d]
};
int64_t rotate_groups(int64_t n_rows);
hipError_t launch_rotate(const RotateArgs& a, bool back, hipStream_t s);

struct CacheArgs {
    int32_t n; const int32_t* page; const int32_t* entry;
    void* st; int64_t st_stride; int32_t n_pages, bf16, vec;
    int8_t* q; float* scale; int32_t n_entries;
    int64_t rows; int32_t dv;    // rows of an entry (heads * d_k) and their width
    int32_t* err;
};
hipError_t launch_cache(const CacheArgs& a, bool store, hipStream_t s);

}  // namespace gdnl
