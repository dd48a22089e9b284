/*
 * gdn_train.h -- the second header of libgdn: the vector-state gated linear
 * recurrence (serving and training form), its backward pass with or without
 * 8-bit checkpoints, and the backward pass of the causal conv of gdn.h.
 *
 * The vector-state recurrence is the layer core of gdn.h with one state value
 * and one pair of gates per channel in place of a d_k x d_v matrix and one
 * pair per head.  Per sequence and channel c, with the gate formulas of
 * gdn.h:
 *     z_t = a_t + dt_bias,  g_t = -exp(A_log) * softplus(z_t),
 *     beta_t = sigmoid(b_t),
 *     h_t = e^{g_t} h_{t-1} + beta_t x_t,
 * h_0 the state page (zero where has_init is 0).
 *
 * Conventions are those of gdn.h: device pointers, caller-owned buffers, no
 * allocation, no synchronisation, no state kept between calls, launches on
 * `stream`, GDN_* status codes and dtypes, GDN_DEVERR_* bits OR-ed into *err.
 * Beyond them:
 * - Rows are packed: row r of x, a, b, h and of every gradient belongs to the
 *   sequence s with cu_seqlens[s] <= r < cu_seqlens[s+1].  Rows of no
 *   sequence (before the first, behind the last) and rows of padding
 *   sequences (page_idx < 0) are neither read nor written.
 * - A sequence is skipped, as a padding one is, and a bit is set, when its
 *   page index is beyond a pool it uses (GDN_DEVERR_PAGE; a backward call knows
 *   state_in alone, so where state_out has fewer pages give it that number in
 *   state_in.n_pages), when its bounds are negative, decreasing, beyond n_rows
 *   or before the end of an earlier valid sequence, or when it is longer than a
 *   max_seqlen > 0 (GDN_DEVERR_BATCH).
 * - Sequences of length 0 are no-ops, whose page stays as it is; a backward
 *   pass hands the gradient of their final state or window through to the
 *   initial one, whatever has_init says.
 * - Any row stride from channels to 2^24 and any element-aligned pointer is
 *   accepted.  Rows on whole vectors are faster: on 16 bytes and in channels a
 *   multiple of 8 for the backward pass of the recurrence in bf16 (by 1.4), on
 *   four elements and in channels a multiple of 4 for the conv and the
 *   one-launch form (by 1.1 to 1.2).
 * - GDN_ERR_ARG, also from the queries, where a kernel would need more threads
 *   than one launch has (2^32): with 128 or fewer channels beyond 2^30 rows, in
 *   general where blocks of 128 rows by 128 channels (or 256 by 64) number 2^23.
 * - Inputs and outputs of one call must not overlap, but a state pool may be
 *   both state_in and state_out.
 * - workspace: 256-byte aligned device memory of at least the queried size,
 *   ignored on entry, scratch on return.  The size queried for a number of
 *   rows serves every call with the same dims and no more rows.  Calls that
 *   share one workspace must be ordered (same stream, or events); graphs
 *   captured over one workspace likewise.
 * - An infinite a or b stands for its limit (e^g and beta are 0 or 1, with no
 *   gradient through them).
 * - All arithmetic is fp32 (sums over rows of a parameter's gradient: fp32
 *   within 256 rows, fp64 across them); results do not depend on timing.  A
 *   state that is not finite stays so to the end of its sequence, whether as
 *   Inf or NaN is not specified.
 * - Every call can be captured in a HIP graph and replayed.
 */
#ifndef GDN_TRAIN_H
#define GDN_TRAIN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Packed rows between two states kept for the backward pass. */
#define GDNT_SCAN_BLOCK 256
/* Rows and channels of a block of the 8-bit checkpoint. */
#define GDNT_CKPT_ROWS 16
#define GDNT_CKPT_CHANNELS 4

/* Sticky device error bit beside those of gdn.h: a wait inside a kernel ran
 * into its bound and the call's results are not valid.  What the wait was for
 * counts as NaN, so the rows, states and gradients that hang on it are NaNs,
 * also where err is NULL. */
#define GDNT_DEVERR_TIMEOUT 32u

typedef struct gdnt_scan_dims {
    int32_t channels;      /* 1 .. 2^24 */
    int32_t act_dtype;     /* x, a, b, h and their gradients: GDN_BF16 or GDN_F32 */
    int32_t state_dtype;   /* state pages: GDN_F32 or GDN_BF16 */
} gdnt_scan_dims;

typedef struct gdnt_scan_params {
    const float* a_log;    /* [channels] */
    const float* dt_bias;  /* [channels] */
} gdnt_scan_params;

/* ------------------------------------------------------------ queries */

/* Bytes of workspace gdnt_scan_forward and gdnt_scan_backward need for a
 * batch of up to n_rows rows (the same for both; host-only). */
int32_t gdnt_scan_workspace_bytes(const gdnt_scan_dims* dims, int32_t n_seqs, int64_t n_rows, size_t* out_bytes);

/* Bytes of what a forward call keeps for its backward call (host-only):
 * *states_bytes for the kept states, fp32 [ceil(n_rows/256)][channels], and
 * *ckpt_bytes for the 8-bit checkpoint.  Either pointer may be NULL. */
int32_t gdnt_scan_saved_bytes(const gdnt_scan_dims* dims, int64_t n_rows, size_t* states_bytes, size_t* ckpt_bytes);

/* Bytes of workspace gdnt_conv_backward needs for a batch of up to n_rows
 * rows (host-only). */
int32_t gdnt_conv_workspace_bytes(const gdn_dims* dims, int32_t n_seqs, int64_t n_rows, size_t* out_bytes);

/* ------------------------------------------- gated linear recurrence */

/* h [n_rows][h_stride] (act dtype) of the recurrence above, and each
 * sequence's last h in its page of state_out (state dtype).  The initial
 * state is read from the same page index of state_in.  A state page holds
 * `channels` values; pool page strides are in elements.
 *   x: [n_rows][x_stride]; a, b: [n_rows][ab_stride].
 * states (NULL, or gdnt_scan_saved_bytes, 16-byte aligned): receives the
 * state before every packed row that is a multiple of GDNT_SCAN_BLOCK and
 * continues a sequence; what gdnt_scan_backward needs beside its inputs.
 * ckpt (NULL, or gdnt_scan_saved_bytes, 256-byte aligned; needs states):
 * receives x, a and b in 8 bits.  Over each block of GDNT_CKPT_ROWS packed
 * rows (from a multiple of it) and GDNT_CKPT_CHANNELS channels, of the rows
 * that belong to a sequence: m = max |v|, up = fl(127 / m), scale =
 * fl(m / 127), q = v * up rounded once to the nearest integer, ties to even;
 * the stored value is q * scale (finite also where m is the largest number:
 * a scale whose 127-fold is not finite counts as the next one below it).  A
 * block with m < 2^-100 is stored as zeros, one with an Inf or NaN as NaNs.
 * Layout, with nb = ceil(n_rows/16) and n4 = ceil(channels/64)*16: int8
 * q[nb][3][n4][16][4] (tensor x, a, b; row and channel within the block
 * innermost), then fp32 scale[nb][3][n4].
 * Batches of at most 4096 sequences with 0 < max_seqlen <= 8 that keep
 * nothing are computed by one launch, others by two. */
int32_t gdnt_scan_forward(const gdnt_scan_dims* dims, const gdnt_scan_params* params,
                          const void* x, int64_t x_stride, const void* a, const void* b, int64_t ab_stride,
                          const gdn_batch* batch, gdn_state_pool state_in, gdn_state_pool state_out,
                          void* h, int64_t h_stride, float* states, void* ckpt,
                          void* workspace, size_t ws_bytes, int32_t* err, void* stream);

/* The gradients of gdnt_scan_forward.  dh [n_rows][dh_stride] (act dtype) is
 * the gradient of h, d_state [n_seqs][channels] fp32 (or NULL: zero) that of
 * the final states before their rounding.  With lambda_t = dh_t +
 * e^{g_{t+1}} lambda_{t+1} (+ d_state at the last row):
 *   dx_t = beta_t lambda_t,  db_t = lambda_t x_t beta_t (1 - beta_t)
 *   (1 - beta_t from beta_t in fp32: within 2^-23 of 1, so that db of a b far
 *   above 0 is small without being exact to its own digits),
 *   dg_t = lambda_t e^{g_t} h_{t-1},  da_t = -exp(A_log) dg_t sigmoid(z_t),
 *   d_dt_bias = sum_t da_t,  d_a_log = sum_t dg_t g_t,
 *   d_state0 = e^{g_1} lambda_1,
 * roundings to the state dtype and act dtype counted as the identity.
 * x, a, b: those of the forward call, or all three NULL and ckpt what the
 * forward call stored; the gradients are then taken at the stored values,
 * with h_{t-1} recomputed from them and from the kept states.  states: what
 * the forward call kept.  state_in: the pages as they were before the
 * forward call (keep a copy where that call worked in place).
 * dx: [n_rows][dx_stride]; da, db: [n_rows][dab_stride] (act dtype);
 * d_a_log, d_dt_bias: [channels] fp32, over the sequences of this call,
 * overwritten (zeros for an empty batch); d_state0: [n_seqs][channels] fp32
 * or NULL, zeros where has_init is 0 (of sequences with rows) and for padding
 * and skipped sequences. */
int32_t gdnt_scan_backward(const gdnt_scan_dims* dims, const gdnt_scan_params* params,
                           const void* x, int64_t x_stride, const void* a, const void* b, int64_t ab_stride,
                           const void* ckpt, const gdn_batch* batch, gdn_state_pool state_in, const float* states,
                           const void* dh, int64_t dh_stride, const float* d_state,
                           void* dx, int64_t dx_stride, void* da, void* db, int64_t dab_stride,
                           float* d_a_log, float* d_dt_bias, float* d_state0,
                           void* workspace, size_t ws_bytes, int32_t* err, void* stream);

/* -------------------------------------------------- conv, backward pass */

/* The gradients of gdn_conv_update (same dims, conv_w, x, batch and
 * activation).  dy [n_rows][dy_stride] (dy_dtype) is the gradient of y;
 * d_window [n_seqs][conv_w-1][C_conv] fp32 (or NULL: zero) that of the rolled
 * windows.  conv holds the windows as they were before the forward call
 * (which rolls them in place: keep a copy); its sync words are not used, and
 * base may be NULL when no sequence of the batch has an initial window
 * (has_init all 0).  With z and X as there and dz_t = dy_t * SiLU'(z_t)
 * (dy_t without activation):
 *   dX_t = sum_j conv_w[c][j] dz_{t+W-1-j},  d_conv_w[c][j] = sum_t dz_t X_{t-W+1+j}.
 * dx: [n_rows][dx_stride] act dtype; d_conv_w: [C_conv][conv_w] fp32, over
 * the sequences of this call, overwritten (zeros for an empty batch);
 * d_window0: [n_seqs][conv_w-1][C_conv] fp32 or NULL, zeros where has_init is
 * 0 (of sequences with rows) and for padding and skipped sequences. */
int32_t gdnt_conv_backward(const gdn_dims* dims, const void* conv_w, const void* x, int64_t x_stride,
                           const void* dy, int32_t dy_dtype, int64_t dy_stride,
                           const gdn_batch* batch, gdn_conv_pool conv, int32_t activation, const float* d_window,
                           void* dx, int64_t dx_stride, float* d_conv_w, float* d_window0,
                           void* workspace, size_t ws_bytes, int32_t* err, void* stream);

#ifdef __cplusplus
}
#endif
#endif
