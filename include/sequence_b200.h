/*
 * sequence_b200.h -- C ABI of the operators over sequences: the causal depthwise
 * convolution over time and the gated linear recurrence, each with its forward pass, its
 * backward pass and its form for one token.
 *
 * The conventions of conv2d_b200.h hold (device pointers, streams, dtypes, statuses,
 * conv2d_last_error, conv2d_sync_status), with these additions:
 *
 * - A tensor over sequences is a matrix of `rows` rows of C channels.  Channels are
 *   contiguous; rows lie `*_stride` elements apart (at least C for what is written; 0 is
 *   allowed for what is read).  Pointers need the alignment of their element only.  Fastest
 *   are tensors whose pointers and row strides are all multiples of 16 bytes (for the
 *   convolution C and the states' pointers multiples of 4 channels too, 2 where K > 4);
 *   others take up to twice the time.
 * - offsets = NULL: the rows are nseq sequences of T rows, rows = nseq * T.  Otherwise
 *   offsets holds nseq + 1 device ints, offsets[0] = 0, never falling, at most `rows`:
 *   sequence s has rows offsets[s] .. offsets[s+1]-1 (it may be empty) and T is ignored.
 *   Rows from offsets[nseq] on belong to no sequence: nothing is read from them into a
 *   result and no output row is written there.  Offsets that break the rule are reported
 *   as CONV_ERR_INVALID_ARG by conv2d_sync_status (the results are then undefined).
 * - A sequence sees only its own rows: infinities and NaN of one never reach another.
 *   Inside it a NaN in a row of the recurrence reaches every later state; an infinite state
 *   leaves infinities or NaN.
 * - Results do not depend on timing: equal inputs give equal bits.
 * - Outputs must not overlap inputs or each other; rows may interleave in one buffer.
 * - rows = 0 is allowed (tensors over rows may then be NULL), nseq = 0 is not.
 * - CONV_ERR_UNSUPPORTED: more than 2^30 rows or channels, or more blocks than one launch takes.
 */
#ifndef SEQUENCE_B200_H
#define SEQUENCE_B200_H

#include "conv2d_b200.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { CONV_ACT_NONE = 0, CONV_ACT_SILU = 1 } conv_activation_t;

/* -------------------------------------- causal depthwise convolution over time ---
 *     z[t][c] = bias[c] + sum_{k < K} w[c][k] * x[t - K + 1 + k][c]
 *     y = z (CONV_ACT_NONE) or z / (1 + exp(-z)) (CONV_ACT_SILU)
 * with t counted inside each sequence: the depthwise convolution (groups = C_in = C_out) of
 * one spatial dimension, padded with K - 1 rows on the left only.  The rows before a
 * sequence are the K - 1 rows of its window in `state`, or zeros.  2 <= K <= 8.  Sums run
 * in fp32 and are rounded once. */

/* The forward pass.
 *   w           : (C, K), dtype          bias : (C,), dtype, or NULL
 *   state       : (nseq, K-1, C), dtype: the rows before each sequence, or NULL (zeros)
 *   final_state : (nseq, K-1, C), or NULL; receives the last K-1 rows of (state, x), the
 *                 window that continues the sequence.  Not `state` itself.  */
int conv1d_causal_forward(const void *x, const void *w, const void *bias, void *y, const void *state,
                          void *final_state, const int *offsets, int nseq, int T, long long rows, int C,
                          int K, conv_activation_t activation, long long x_stride, long long y_stride,
                          conv_dtype_t dtype, conv_stream_t stream);

/* Device scratch bytes of conv1d_causal_backward on the current device. */
int conv1d_causal_backward_workspace_size(long long rows, int C, int K, size_t *bytes);

/* The backward pass, from the forward pass's inputs and dy = dL/dy.
 *   d_final_state : dL/dfinal_state, (nseq, K-1, C), or NULL (zeros)
 *   dx, dw, db, d_state : gradients in dtype (summed in fp32, rounded once); db and d_state may be NULL */
int conv1d_causal_backward(const void *x, const void *w, const void *bias, const void *dy, const void *state,
                           const void *d_final_state, void *dx, void *dw, void *db, void *d_state,
                           const int *offsets, int nseq, int T, long long rows, int C, int K,
                           conv_activation_t activation, long long x_stride, long long dy_stride,
                           long long dx_stride, conv_dtype_t dtype, void *workspace, size_t workspace_bytes,
                           conv_stream_t stream);

/* One token for each of B sequences: x and y have B rows, and the windows state[slot]
 * (pool of (K-1, C) windows) move on by that row in place.  slots: B device ints, or NULL
 * (row b has window b; pool >= B).  A slot outside [0, pool) marks a row without a sequence:
 * its y is left as it was.  Two rows must not name the same slot: the later one is then left
 * out and conv2d_sync_status reports CONV_ERR_INVALID_ARG. */
int conv1d_causal_step(const void *x, const void *w, const void *bias, void *y, void *state, const int *slots,
                       int B, int pool, int C, int K, conv_activation_t activation, long long x_stride,
                       long long y_stride, conv_dtype_t dtype, conv_stream_t stream);

/* --------------------------------------------------- gated linear recurrence ---
 *     ra = sigmoid(gate_a[t][c]),  rx = sigmoid(gate_x[t][c])
 *     a  = exp(-kappa * softplus(decay[c]) * ra)
 *     h[t][c] = a * h[t-1][c] + sqrt(1 - a^2) * rx * x[t][c]
 * with h before a sequence taken from `state`, or zero.  decay and all states are fp32
 * whatever the dtype; h is carried in fp32 and rounded once into y.  Where a is 1 to within
 * 1e-37 (gate_a of the lowest value, or -infinity) the row keeps the state and adds
 * 0 * rx * x.  kappa: finite and above 0. */

/* Bytes of the states that the forward pass saves for the backward pass (opaque): an fp32 state
 * for every 8 rows, an eighth of the bytes of y in fp32 and a quarter in bf16.  T = 0: packed
 * sequences (here and below). */
int gated_recurrence_saved_size(int nseq, int T, long long rows, int C, conv_dtype_t dtype, size_t *bytes);

/* Device scratch bytes of the forward pass, and of the backward pass. */
int gated_recurrence_workspace_size(int nseq, int T, long long rows, int C, conv_dtype_t dtype, size_t *bytes);
int gated_recurrence_backward_workspace_size(int nseq, int T, long long rows, int C, conv_dtype_t dtype, size_t *bytes);

/* The forward pass: y = h.
 *   state, final_state : (nseq, C) fp32, or NULL; final_state receives the last h of each
 *                        sequence (its state where it is empty).  Not `state` itself.
 *   saved              : gated_recurrence_saved_size() bytes for a backward pass, or NULL */
int gated_recurrence_forward(const void *x, const void *gate_a, const void *gate_x, const float *decay,
                             float kappa, void *y, const float *state, float *final_state, void *saved,
                             const int *offsets, int nseq, int T, long long rows, int C, long long x_stride,
                             long long gate_a_stride, long long gate_x_stride, long long y_stride,
                             conv_dtype_t dtype, void *workspace, size_t workspace_bytes, conv_stream_t stream);

/* The backward pass, from the forward pass's inputs, its `saved` and dy = dL/dy.
 *   d_final_state              : dL/dfinal_state, (nseq, C) fp32, or NULL (zeros)
 *   dx, d_gate_a, d_gate_x     : dtype
 *   d_decay (C,), d_state (nseq, C) or NULL : fp32 */
int gated_recurrence_backward(const void *x, const void *gate_a, const void *gate_x, const float *decay,
                              float kappa, const void *dy, const void *saved, const float *state,
                              const float *d_final_state, void *dx, void *d_gate_a, void *d_gate_x,
                              float *d_decay, float *d_state, const int *offsets, int nseq, int T,
                              long long rows, int C, long long x_stride, long long gate_a_stride,
                              long long gate_x_stride, long long dy_stride, long long dx_stride,
                              long long d_gate_a_stride, long long d_gate_x_stride, conv_dtype_t dtype,
                              void *workspace, size_t workspace_bytes, conv_stream_t stream);

/* One token for each of B sequences; state (pool of C fp32 values) is updated in place, slots as in
 * conv1d_causal_step. */
int gated_recurrence_step(const void *x, const void *gate_a, const void *gate_x, const float *decay, float kappa,
                          void *y, float *state, const int *slots, int B, int pool, int C, long long x_stride,
                          long long gate_a_stride, long long gate_x_stride, long long y_stride,
                          conv_dtype_t dtype, conv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SEQUENCE_B200_H */
