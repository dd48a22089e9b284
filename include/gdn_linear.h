/*
 * gdn_linear.h -- the third header of libgdn: linear attention with a decay
 * for each head (the matrix-state recurrence of gdn.h without its delta
 * correction), forward and backward; the norms of queries and keys for each
 * head with the rotation by position in front of it; and state pages kept in
 * 8 bits.
 *
 * Per sequence and value head h, with key head h / (h_v/h_k):
 *     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,
 * S a d_k x d_v matrix, S_0 the state page (zero where has_init is 0), g the
 * log decay of a row and value head, or one for each value head.
 *
 * Conventions are those of gdn.h: device pointers, caller-owned buffers, no
 * allocation, no synchronisation, no state kept between calls, launches on
 * `stream`, GDN_* status codes and dtypes, GDN_DEVERR_* bits OR-ed into *err,
 * state pages of h_v row-major d_k x d_v matrices.  Beyond them:
 * - Rows are packed: row r belongs to the sequence s with cu_seqlens[s] <= r <
 *   cu_seqlens[s+1].  Rows of no sequence and rows of padding sequences
 *   (page_idx < 0) are neither read nor written.
 * - A sequence is skipped, as a padding one is, and a bit is set, when its page
 *   index is beyond a pool it uses (GDN_DEVERR_PAGE; a backward call knows
 *   state_in alone), when its bounds are negative, decreasing, beyond n_rows or
 *   before the end of an earlier valid sequence, or when it is longer than a
 *   max_seqlen > 0 (GDN_DEVERR_BATCH).
 * - Sequences of length 0 are no-ops, whose page stays as it is; a backward
 *   pass hands the gradient of their final state through to the initial one,
 *   whatever has_init says.
 * - A row holds its heads one behind the other.  Any row stride from the row's
 *   width to 2^24 and any element-aligned pointer is accepted.  Rows on 16 bytes
 *   whose heads are a multiple of 16 bytes wide are faster.
 * - Inputs and outputs of one call must not overlap, but a state pool may be
 *   both state_in and state_out.
 * - workspace: 256-byte aligned device memory of at least the queried size,
 *   ignored on entry, scratch on return.  The size queried serves every call
 *   with the same dims, no more sequences and no more rows.  Calls that share
 *   one workspace must be ordered (same stream, or events); graphs captured
 *   over one workspace likewise.
 * - Sums, states and softly decayed weights are held in fp32 or more; results
 *   do not depend on timing.
 * - Every call can be captured in a HIP graph and replayed.
 * - Limits, beyond which a call is refused with GDN_ERR_ARG before anything is
 *   launched: n_rows up to 2^31 - 1025, n_seqs up to 2^28, a pool of up to
 *   2^29 - 1 pages, h_v d_k and h_v d_v up to 2^24, a state of up to 2^31 values.
 *   A launch has 2^23 - 1 workgroups: row by row one for a sequence and value
 *   head; in chunks one for a segment and value head, of which a batch has up to
 *   n_seqs + n_rows / 128 + 2, at most n_seqs + 512 / h_v + 2 (backward: or
 *   n_seqs + n_rows / 2048 + 2, where that is more), and 7 more for each head of
 *   a key head's; in a call on 8-bit entries one for a pair and 64 blocks of
 *   GDNL_CACHE_COLS columns.  262,000 sequences of 32 heads are within them.
 */
#ifndef GDN_LINEAR_H
#define GDN_LINEAR_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdnl_dims {
    int32_t h_k, h_v;      /* key heads (of q and k), value heads; h_v % h_k == 0 */
    int32_t d_k, d_v;      /* head dims, 1 .. 128 for the attend calls */
    int32_t act_dtype;     /* q, k, v, o and their gradients: GDN_BF16 or GDN_F32 */
    int32_t state_dtype;   /* state pages: GDN_F32 or GDN_BF16 */
    float scale;
} gdnl_dims;

/* Columns of a state's row that share one scale in an 8-bit entry. */
#define GDNL_CACHE_COLS 64

/* Norms of gdnl_rotate_*: x / sqrt(mean x^2 + eps), or x / sqrt(sum x^2 + eps). */
#define GDNL_NORM_RMS 0
#define GDNL_NORM_L2 1
/* Pairs that are rotated: value i with value i + rot/2, or 2i with 2i + 1. */
#define GDNL_PAIRS_HALVES 0
#define GDNL_PAIRS_NEIGHBOURS 1

/* ------------------------------------------------- linear attention */

/* Batches with 0 < max_seqlen <= this are computed row by row. */
#define GDNL_TOKEN_ROWS 8

/* What a backward call is asked for and given: dg, d_state, d_state0. */
#define GDNL_ASKS 16
#define GDNL_ASKS_DG 1
#define GDNL_ASKS_D_STATE 2
#define GDNL_ASKS_D_STATE0 4

/* Bytes of workspace gdnl_attend_forward (backward = 0) or
 * gdnl_attend_backward (1) needs for a batch of up to n_seqs sequences and
 * n_rows rows (host-only).  backward = GDNL_ASKS, or-ed with GDNL_ASKS_* for
 * those of the three arguments that are not NULL: for such calls alone, a state
 * for every sequence less where no dg is wanted, where there is no d_state, or
 * where d_state0 is given. */
int32_t gdnl_attend_workspace_bytes(const gdnl_dims* dims, int32_t n_seqs, int64_t n_rows, int32_t backward,
                                    size_t* out_bytes);

/* o of the recurrence above, and each sequence's last state in its page of
 * state_out.  The initial state is read from the same page index of state_in.
 *   q, k: [n_rows][stride >= h_k*d_k], v, o: [n_rows][stride >= h_v*d_v] act
 *   dtype; g: fp32 [n_rows][g_stride >= h_v], or with g_stride 0 [h_v], the
 *   decays of every row.
 * A g below -128 counts as a decay of exactly 0 (so an infinite one begins a
 * sequence anew); NaN stays NaN.  A value that is not finite reaches its own
 * column of o and of the state from its row on and nothing before that.
 * Batches with 0 < max_seqlen <= GDNL_TOKEN_ROWS are computed row by row in one
 * launch without a workspace, others, whatever the lengths of their shorter
 * sequences, in chunks of 64 rows on matrix cores. */
int32_t gdnl_attend_forward(const gdnl_dims* dims, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const float* g, int64_t g_stride,
                            const gdn_batch* batch, gdn_state_pool state_in, gdn_state_pool state_out,
                            void* o, int64_t o_stride, void* workspace, size_t ws_bytes, int32_t* err, void* stream);

/* The gradients of gdnl_attend_forward.  d_o [n_rows][do_stride] (act dtype)
 * is the gradient of o, d_state [n_seqs][h_v][d_k][d_v] fp32 (or NULL: zero)
 * that of the final states before their rounding.  With E_t = e^{g_{t+1}}
 * E_{t+1} + scale q_t d_o_t^T (+ d_state at the last row):
 *   dq_t = scale S_t d_o_t, dk_t = E_t v_t  (summed over the value heads of a
 *   key head),  dv_t = E_t^T k_t,  dg_t = e^{g_t} <S_{t-1}, E_t>,
 *   d_state0 = e^{g_1} E_1,
 * roundings to the state dtype and act dtype counted as the identity; nothing
 * of the forward call is kept.  state_in: the pages as they were before the
 * forward call (keep a copy where that call worked in place).
 * dg: fp32 [n_rows][h_v], or [h_v] with g_stride 0: the sum over the rows of
 * this call's sequences (zeros for an empty batch); NULL: not wanted.  Where g
 * is below -128 its gradient is 0.  d_state0: [n_seqs][h_v][d_k][d_v] fp32 or
 * NULL, zeros where has_init is 0 (of sequences with rows) and for padding and
 * skipped sequences.  Inputs that are not finite leave gradients of their own
 * sequence unspecified, and none of another's (but for a dg of [h_v]). */
int32_t gdnl_attend_backward(const gdnl_dims* dims, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const float* g, int64_t g_stride,
                             const gdn_batch* batch, gdn_state_pool state_in, const void* d_o, int64_t do_stride,
                             const float* d_state, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                             void* dv, int64_t dv_stride, float* dg, float* d_state0,
                             void* workspace, size_t ws_bytes, int32_t* err, void* stream);

/* --------------------------------- head norms and rotation by position */

typedef struct gdnl_rotate_dims {
    int32_t h_q, h_k;      /* heads of a row of q and of k (either may be 0) */
    int32_t d;             /* head dim, even, 2 .. 256 */
    int32_t rot;           /* leading values of a head that are rotated: even, 0 .. d */
    int32_t act_dtype;     /* GDN_BF16 or GDN_F32 */
    int32_t norm;          /* GDNL_NORM_* */
    int32_t pairs;         /* GDNL_PAIRS_* */
    float eps;             /* >= 0 */
} gdnl_rotate_dims;

/* Bytes of workspace gdnl_rotate_backward needs for up to n_rows rows (host-only). */
int32_t gdnl_rotate_workspace_bytes(const gdnl_rotate_dims* dims, int64_t n_rows, size_t* out_bytes);

/* For every head x of a row: n = x / sqrt(mean or sum of x^2 + eps) * w, then
 * the first `rot` values turned in pairs by the angle pos * inv_freq[i]:
 *   (a, b) -> (a cos - b sin, b cos + a sin),
 * the angle taken in 64 bits, the rest in fp32, one rounding at the end; the
 * norm is a number for every head of numbers, the largest and smallest too.
 *   q, yq: [n_rows][stride >= h_q*d]; k, yk: [n_rows][stride >= h_k*d] act
 *   dtype; wq, wk: fp32 [d] or NULL (ones); pos: int32 [n_rows]; inv_freq:
 *   fp32 [rot/2].
 * yq may be q and yk may be k, with the same stride. */
int32_t gdnl_rotate_forward(const gdnl_rotate_dims* dims, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const float* wq, const float* wk, const int32_t* pos,
                            const float* inv_freq, int64_t n_rows, void* yq, int64_t yq_stride, void* yk,
                            int64_t yk_stride, void* stream);

/* The gradients of gdnl_rotate_forward from those of yq and yk: dq and dk (act
 * dtype; dq may be d_yq and dk may be d_yk, with the same stride), dwq and dwk
 * fp32 [d] or NULL, summed over rows and heads, overwritten (zeros for no
 * rows). */
int32_t gdnl_rotate_backward(const gdnl_rotate_dims* dims, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const float* wq, const float* wk, const int32_t* pos,
                             const float* inv_freq, int64_t n_rows, const void* d_yq, int64_t d_yq_stride,
                             const void* d_yk, int64_t d_yk_stride, void* dq, int64_t dq_stride, void* dk,
                             int64_t dk_stride, float* dwq, float* dwk, void* workspace, size_t ws_bytes,
                             void* stream);

/* ------------------------------------------- state pages in 8 bits */

/* Entries of state pages in 8 bits: q int8 [n_entries][h_v][d_k][d_v] and
 * scale fp32 [n_entries][h_v][d_k][ceil(d_v/64)].  Over each GDNL_CACHE_COLS
 * columns of a row (the last block may have fewer): m = max |v|, up =
 * fl(127 / m), scale = fl(m / 127), q = v * up rounded once to the nearest
 * integer, ties to even; the stored value is q * scale.  A block with m <
 * 2^-100 is stored as zeros, one with an Inf or NaN as NaNs; a scale whose
 * 127-fold is not finite counts as the next one below it.  State pages are
 * those of the attend calls and of gdn.h: any d_k and d_v. */
typedef struct gdnl_cache {
    int8_t* q;             /* 4-byte aligned */
    float* scale;
    int32_t n_entries;
} gdnl_cache;

/* Bytes of q and of scale for n_entries entries (host-only).  Either pointer may be NULL. */
int32_t gdnl_cache_bytes(const gdnl_dims* dims, int32_t n_entries, size_t* q_bytes, size_t* scale_bytes);

/* Entry entry[i] <- state page page_idx[i], for i < n.  An index < 0 in either
 * skips the pair; a page beyond the pool (GDN_DEVERR_PAGE) or an entry beyond
 * the cache (GDN_DEVERR_CACHE) does so with its bit set.  Entries of one call
 * must be distinct (pages may repeat). */
int32_t gdnl_cache_store(const gdnl_dims* dims, int32_t n, const int32_t* page_idx, const int32_t* entry,
                         gdn_state_pool state, const gdnl_cache* cache, int32_t* err, void* stream);

/* State page page_idx[i] <- entry entry[i], in the state dtype.  Pages of one
 * call must be distinct (entries may repeat). */
int32_t gdnl_cache_load(const gdnl_dims* dims, int32_t n, const int32_t* entry, const int32_t* page_idx,
                        const gdnl_cache* cache, gdn_state_pool state, int32_t* err, void* stream);

#ifdef __cplusplus
}
#endif
#endif
