/*
 * convseq.h -- C ABI of the sequence operators of the channels-last
 * convolution library for AMD Instinct MI355X (gfx950): what a recurrent block
 * puts around its projections (1x1 convolutions of convfwd.h).
 *
 *   - causal depthwise convolution along a sequence, with bias, activation and
 *     carried rows: forward, backward and single-row step;
 *   - gated linear recurrence over a sequence: forward, backward and
 *     single-row step;
 *   - activations kept in 8 bits between the forward and the backward pass,
 *     written by the two forward passes as they read their inputs (or by
 *     convseq_pack8) and read by the two backward passes (or convseq_unpack8).
 *
 * Layouts.  A sequence tensor is (B, T, C), channels fastest.  Inputs marked
 * "rows" may be views: channel stride 1, any batch and row stride >= 0 in
 * elements (a column slice of a wider projection, an expanded tensor).
 * Everything else, and every output, is dense.
 *
 * dtype (convfwd_dtype) is the type of sequence tensors and of the
 * convolution's filter, bias and carried rows.  The recurrence's state, its
 * log-decay parameter, every gradient of a parameter or state of the
 * recurrence, and the filter's and bias's gradients are fp32.  All arithmetic
 * is fp32; results are rounded once, to nearest even.  Sums over rows are
 * added in a fixed order: the same call gives the same bits.
 *
 * starts (B, T), bytes, may be NULL: a nonzero byte marks a row that begins a
 * new sequence.  Nothing, NaN and infinities included, crosses a start, and a
 * start at row 0 shuts out the carried rows or state.  What a backward pass reads
 * in 8 bits was made in groups of 16 rows that no start divides: there the
 * sequences that share a group also share its power of two, and a NaN or an
 * infinity in it makes all of its rows NaN, on both sides of a start.
 *
 * Ownership, streams and errors are those of convfwd.h: the caller owns every
 * buffer (workspaces included; their sizes come from the *_workspace calls,
 * they need 16-byte alignment, no initial contents, and must not be shared by
 * calls that may run at the same time), nothing is allocated or synchronised,
 * launches go to `stream`, arguments are validated before the GPU is touched,
 * and the calls may be captured into a graph.  Outputs may overlap no other
 * buffer of the call (the step calls' state excepted).  Pointers must be
 * aligned to their element.  B = 0 and T = 0 are valid: outputs over rows are
 * empty, parameter gradients are zero, carried rows and states pass through.
 */
#ifndef CONVSEQ_H
#define CONVSEQ_H

#include <stdint.h>

#include "convfwd.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  CONVSEQ_STATE_ROWS = 64, /* rows between the recurrence's kept states */
  CONVSEQ_GROUP_ROWS = 16  /* rows of a channel that share a power of two in 8 bits */
};

typedef enum { CONVSEQ_ACT_NONE = 0, CONVSEQ_ACT_SILU = 1 } convseq_act;

/* A (B, T, C) input with channel stride 1. */
typedef struct {
  const void* data;
  int64_t batch_stride, row_stride; /* elements, >= 0 */
} convseq_rows;

/* A (B, T, C) tensor in 8 bits: 16 consecutive rows t of a channel (the last
 * group may be short) share the byte e[b, t/16, c], and the value held at
 * (b, t, c) is q[b, t/16, t%16/8, c, t%8] * 2^(e - 127).  With M the largest magnitude
 * of the group, e - 127 = max(floor(log2 M) - 6, -126) and q is x / 2^(e - 127)
 * rounded to nearest even within +-127.  A group that contains an infinity or
 * a NaN has e = 255 and is read back as NaN throughout, whatever starts lie in
 * it.  q (B, ceil(T/16), 2,
 * C, 8) and e (B, ceil(T/16), C) are dense and q is 16-byte aligned; rows past
 * T are written as zero. */
typedef struct {
  void* q; /* int8, 16-byte aligned */
  void* e; /* uint8 */
} convseq_kept;

typedef struct {
  int32_t b, t, c;
  int32_t k;     /* taps, 1..8 */
  int32_t act;   /* convseq_act */
  int32_t dtype; /* convfwd_dtype */
} convseq_conv_desc;

/* z[b,t,c] = bias[c] + sum_k w[c,k] * X(b, t - (K-1) + k, c),  y = z or z * sigmoid(z)
 *
 * X(b, s, c) is x[b,s,c], for s < 0 the carried row state[b, s + K-1, c]
 * (zeros if state is NULL), and zero where a start lies in (s, t].  w (C, K)
 * (the depthwise filter (C_out, 1, K, 1) of convfwd.h with its unit extents
 * dropped; convfwd.h's grouped path with a low pad of K-1 computes the same z
 * without bias, carried rows and starts, 1.3 to 2.6 times slower).  state_out (may be NULL) receives the last K-1 of the rows
 * (state, x), those before the last start zeroed: the carried rows of the
 * next piece.  kept (NULL, or both pointers set) receives x in 8 bits. */
int convseq_conv_fwd(const convseq_conv_desc* desc, const convseq_rows* x, const void* w, const void* bias,
                     const void* state, const void* starts, void* y, void* state_out,
                     const convseq_kept* kept, void* stream);

/* Gradients of convseq_conv_fwd.  dy is the gradient of y and dstate_out
 * (B, K-1, C) (may be NULL) that of state_out.  x comes as it was (x) or in
 * 8 bits (kept): exactly one of the two is not NULL.  Outputs: dx (dtype),
 * dw (C, K) and dbias (C) (fp32; dbias may be NULL), dstate (B, K-1, C)
 * (dtype; may be NULL). */
int64_t convseq_conv_bwd_workspace(const convseq_conv_desc* desc); /* bytes, or a negative error */
int convseq_conv_bwd(const convseq_conv_desc* desc, const convseq_rows* dy, const convseq_rows* x,
                     const convseq_kept* kept, const void* w, const void* bias, const void* state,
                     const void* starts, const void* dstate_out, void* dx, void* dw, void* dbias, void* dstate,
                     void* workspace, void* stream);

/* One row of each of B streams (desc->t is not used): y (B, C) from x (B, C)
 * with row stride x_row, and the carried rows moved on by one.  Stream b's
 * carried rows are state[slot, :, :], slot = b, or slots[b] (int32) if slots
 * is not NULL; a slot outside [0, n_slots) marks an idle stream: its y is
 * zero and no state is touched.  The moved-on rows go to state_out at the same
 * slot, which may be state itself.  Where it is another buffer, the slots that no
 * stream names are not copied to it: a caller that swaps the two after each call
 * has to step every stream, or update in place.  Two streams must not share a slot. */
int convseq_conv_step(const convseq_conv_desc* desc, const void* x, int64_t x_row, const void* w,
                      const void* bias, const void* state, void* state_out, const void* slots, int32_t n_slots,
                      void* y, void* stream);

typedef struct {
  int32_t b, t, c;
  int32_t dtype; /* convfwd_dtype */
  float decay;   /* > 0 */
} convseq_scan_desc;

/* r = sigmoid(gate_r), i = sigmoid(gate_i), a = exp(-decay * softplus(lam[c]) * r),
 * h_t = a * h_{t-1} + sqrt(1 - a^2) * i * x_t,  y = h
 *
 * A row at a start is scaled by sqrt(1 - a^2) like any other: h_t = sqrt(1 - a^2) * i * x_t.
 * (There is no form in which the first row of a sequence enters unscaled.)
 * with h_{-1} = h0[b,c] (fp32; zeros if NULL) and h_{t-1} absent at a start.
 * a and its products are positive and count as 2^-149 where fp32 would round
 * them to zero: an infinite state, or state's gradient, stays infinite.
 * y (B, T, C), h_last (B, C) fp32 (may be NULL), states (B, ceil(T/64), C)
 * fp32 (may be NULL): the h before rows 0, 64, 128, ..., from which the
 * backward pass starts each piece.  kept (may be NULL): x, gate_r and gate_i in
 * 8 bits, in this order. */
int64_t convseq_scan_fwd_workspace(const convseq_scan_desc* desc); /* bytes, or a negative error */
int convseq_scan_fwd(const convseq_scan_desc* desc, const convseq_rows* x, const convseq_rows* gate_r,
                     const convseq_rows* gate_i, const void* lam, const void* h0, const void* starts, void* y,
                     void* h_last, void* states, const convseq_kept kept[3], void* workspace, void* stream);

/* Gradients of convseq_scan_fwd.  dy is the gradient of y, dh_last (B, C) fp32
 * (may be NULL) that of h_last.  The inputs come as they were (x, gate_r,
 * gate_i) or in 8 bits (kept[3]): all three one way, the other NULL.  h is
 * computed again piece by piece from states.  Outputs: dx, dgate_r, dgate_i
 * (dtype), dlam (C) and dh0 (B, C) (fp32; dh0 may be NULL). */
int64_t convseq_scan_bwd_workspace(const convseq_scan_desc* desc); /* bytes, or a negative error */
int convseq_scan_bwd(const convseq_scan_desc* desc, const convseq_rows* dy, const convseq_rows* x,
                     const convseq_rows* gate_r, const convseq_rows* gate_i, const convseq_kept kept[3],
                     const void* lam, const void* states, const void* starts, const void* dh_last, void* dx,
                     void* dgate_r, void* dgate_i, void* dlam, void* dh0, void* workspace, void* stream);

/* One row of each of B streams (desc->t is not used): y (B, C) and the moved-on
 * state from rows x, gate_r, gate_i (B, C) with the given row strides.  State
 * (fp32), slots and state_out as for convseq_conv_step. */
int convseq_scan_step(const convseq_scan_desc* desc, const void* x, int64_t x_row, const void* gate_r,
                      int64_t r_row, const void* gate_i, int64_t i_row, const void* lam, const void* state,
                      void* state_out, const void* slots, int32_t n_slots, void* y, void* stream);

/* x (B, T, C) into 8 bits, and back (out (B, T, C), dense, rounded to dtype
 * where dtype cannot hold the value). */
int convseq_pack8(int32_t b, int32_t t, int32_t c, int32_t dtype, const convseq_rows* x,
                  const convseq_kept* kept, void* stream);
int convseq_unpack8(int32_t b, int32_t t, int32_t c, int32_t dtype, const convseq_kept* kept, void* out,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVSEQ_H */
