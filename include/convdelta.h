/*
 * convdelta.h -- C ABI of the gated delta rule of the convolution library for
 * AMD Instinct MI355X (gfx950): the recurrence of convseq.h with a matrix for
 * a state, written by key and read by query.
 *
 * Per batch row b and value head h, whose key head is h / (Hv / Hk), with a
 * state S of (Dk, Dv) and a_t = exp(log_decay[b,t,h]):
 *
 *   S' = a_t S_{t-1}                       (S_{t-1} absent at a start)
 *   x_t = v_t - S'^T k_t,  u_t = beta_t x_t
 *   S_t = S' + k_t u_t^T,  y_t = scale * S_t^T q_t
 *
 * q and k are (B, T, Hk, Dk), v and y (B, T, Hv, Dv), log_decay and beta
 * (B, T, Hv).  q and k enter as they are: a layer brings them to length one
 * itself.  Head inputs may be views: element stride 1 within a head, any head,
 * row and batch stride >= 0 (slices of one projection, expanded tensors).
 * Everything else, and every output, is dense.
 *
 * dtype (convfwd_dtype) is the type of q, k, v, y and their gradients.  States,
 * log_decay, beta and the gradients of those are fp32.  Arithmetic has fp32's
 * precision throughout (sums of log decays within 64 rows are fp64), results are
 * rounded once, to nearest even, and sums are added in a fixed order: the same
 * call gives the same bits.  Values of less than 2^-95 lose bits, and fp32 values of
 * 2^128 - 2^119 or more count as infinities.
 *
 * log_decay may have either sign.  Rows are taken 64 at a time (0 .. 63, 64 ..
 * 127, ...), and errors are relative to what a state would grow to inside them if
 * nothing were subtracted from it: log decays above zero whose sum there is g cost
 * a factor of up to exp(g).  Where that overflows, the forward pass goes row by
 * row, and gradients are not finite.
 *
 * starts (B, T), bytes, may be NULL: a nonzero byte marks a row that begins a
 * new sequence, as in convseq.h.  Nothing, NaN and infinities included, crosses
 * a start.  A decay that is zero in fp32 makes its row a start (its gradient is
 * zero).  In the forward pass a NaN or an infinity reaches no earlier row and,
 * where it came with v, no other column; an infinity may come back as NaN.  In the
 * backward pass it may reach all rows of its sequence within its 64 rows.
 *
 * Ownership, streams, workspaces and errors are those of convseq.h.  B = 0 and
 * T = 0 are valid: the state passes through.  CONVFWD_ERR_TOO_LARGE: Hv * Dv of
 * 2^23 elements, Dv of 2^22, a row stride of v or dy of 2^23, or more, T of 2^30,
 * or 2^23 workgroups of a launch (heads times 64 rows, heads times 16 columns).
 */
#ifndef CONVDELTA_H
#define CONVDELTA_H

#include <stdint.h>

#include "convseq.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  CONVDELTA_STATE_ROWS = 64, /* rows between the kept states */
  CONVDELTA_MAX_DK = 128
};

typedef struct {
  int32_t b, t;
  int32_t hk, hv; /* heads of q and k, and of v; hk divides hv */
  int32_t dk, dv; /* dk <= CONVDELTA_MAX_DK */
  int32_t dtype;  /* convfwd_dtype */
  float scale;    /* finite */
} convdelta_desc;

/* A (B, T, H, D) input with element stride 1; strides in elements, >= 0. */
typedef struct {
  const void* data;
  int64_t batch_stride, row_stride, head_stride;
} convdelta_heads;

/* y (B, T, Hv, Dv), h_last (B, Hv, Dk, Dv) fp32.  h0 (B, Hv, Dk, Dv) fp32 may be
 * NULL: zeros.  For the backward pass, both or neither NULL: states (B, ceil(T/64),
 * Hv, Dk, Dv) fp32, the S before rows 0, 64, 128, ..., and x (B, T, Hv, Dv) fp32. */
int64_t convdelta_fwd_workspace(const convdelta_desc* desc); /* bytes, or a negative error */
int convdelta_fwd(const convdelta_desc* desc, const convdelta_heads* q, const convdelta_heads* k,
                  const convdelta_heads* v, const void* log_decay, const void* beta, const void* h0,
                  const void* starts, void* y, void* h_last, void* states, void* x, void* workspace, void* stream);

/* Gradients of convdelta_fwd.  dy is the gradient of y, dh_last (B, Hv, Dk, Dv)
 * fp32 (may be NULL) that of h_last; the other inputs are the forward pass's, and
 * states and x what it kept.  Outputs: dq, dk (B, T, Hk, Dk), added over the value heads
 * that share a key head before they are rounded, dv (B, T, Hv, Dv) (dtype),
 * dlog_decay and dbeta (B, T, Hv), dh0 (B, Hv, Dk, Dv) (fp32). */
int64_t convdelta_bwd_workspace(const convdelta_desc* desc); /* bytes, or a negative error */
int convdelta_bwd(const convdelta_desc* desc, const convdelta_heads* dy, const convdelta_heads* q,
                  const convdelta_heads* k, const convdelta_heads* v, const void* log_decay, const void* beta,
                  const void* states, const void* x, const void* starts, const void* dh_last, void* dq, void* dk,
                  void* dv, void* dlog_decay, void* dbeta, void* dh0, void* workspace, void* stream);

/* One row of each of B streams (desc->t is not used; row strides are not used):
 * y (B, Hv, Dv) and the moved-on state.  Stream b's state is state[slot], slot =
 * b, or slots[b] (int32) if slots is not NULL; a slot outside [0, n_slots) marks an
 * idle stream: its y is zero and no state is touched.  state (n_slots, Hv, Dk, Dv)
 * fp32; the moved-on state goes to state_out at the same slot, which may be state
 * itself.  Slots that no stream names are not copied to another buffer.  Two
 * streams must not share a slot. */
int convdelta_step(const convdelta_desc* desc, const convdelta_heads* q, const convdelta_heads* k,
                   const convdelta_heads* v, const void* log_decay, const void* beta, const void* state,
                   void* state_out, const void* slots, int32_t n_slots, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVDELTA_H */
