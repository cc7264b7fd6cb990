// seq_api.cpp -- the C ABI declared in include/convseq.h: validation, the
// empty problems and the launches on the caller's stream.  No device memory is
// allocated here and nothing is synchronised.
#include "../../include/convseq.h"

#include <stdint.h>

#include "seq_buffers.h"

using namespace convseq;

namespace {

// Extents and type shared by every call.  A launch over rows has at most one
// workgroup per 16 rows and 64 channels, of at most 512 threads; one over
// channels alone (the sums of the backward passes) 1024 threads per 32 channels
// along x.  Each dimension of a grid holds less than 2^32 threads.
int check_extents(int64_t b, int64_t t, int64_t c, int dtype) {
  if (b < 0 || t < 0 || c < 1) return CONVFWD_ERR_BAD_DESC;
  if (dtype != CONVFWD_F32 && dtype != CONVFWD_F16 && dtype != CONVFWD_BF16) return CONVFWD_ERR_UNSUPPORTED;
  const int64_t blocks = (t + kGroup - 1) / kGroup, cols = (c + 63) / 64;
  const int64_t lim = (int64_t)1 << 22;
  if (c >= (int64_t)1 << 26 || b >= lim || blocks >= lim) return CONVFWD_ERR_TOO_LARGE;
  if (b * (blocks > 0 ? blocks : 1) >= (int64_t)1 << 31 || b * (blocks > 0 ? blocks : 1) * cols >= lim * 2)
    return CONVFWD_ERR_TOO_LARGE;
  return CONVFWD_OK;
}

int check_conv(const convseq_conv_desc* d) {
  if (!d) return CONVFWD_ERR_NULL;
  const int rc = check_extents(d->b, d->t, d->c, d->dtype);
  if (rc < 0) return rc;
  if (d->k < 1 || d->act < 0 || d->act > CONVSEQ_ACT_SILU) return CONVFWD_ERR_BAD_DESC;
  return d->k > kMaxTaps ? CONVFWD_ERR_UNSUPPORTED : CONVFWD_OK;
}

int check_scan(const convseq_scan_desc* d) {
  if (!d) return CONVFWD_ERR_NULL;
  const int rc = check_extents(d->b, d->t, d->c, d->dtype);
  if (rc < 0) return rc;
  // a positive finite number (NaN fails the comparison)
  return d->decay > 0.f && d->decay < 1e30f ? CONVFWD_OK : CONVFWD_ERR_BAD_DESC;
}

}  // namespace

extern "C" {

int convseq_conv_fwd(const convseq_conv_desc* d, const convseq_rows* x, const void* w, const void* bias,
                     const void* state, const void* starts, void* y, void* state_out,
                     const convseq_kept* kept, void* stream) {
  const int rc = check_conv(d);
  if (rc < 0) return rc;
  const int eb = elem_bytes(d->dtype);
  const int64_t n = (int64_t)d->b * d->t * d->c, rows = (int64_t)d->b * (d->k - 1) * d->c;
  ConvArgs a{};
  Buffers buf;
  buf.rows(x, d->b, d->t, d->c, eb, &a.x);
  buf.in(w, (int64_t)d->c * d->k * eb, eb);
  buf.in(bias, (int64_t)d->c * eb, eb, false);
  buf.in(state, rows * eb, eb, false);
  buf.in(starts, (int64_t)d->b * d->t, 1, false);
  buf.out(y, n * eb, eb);
  buf.out(state_out, rows * eb, eb, false);
  buf.kept(kept, d->b, d->t, d->c, true, &a.kept);
  if (buf.result() < 0) return buf.result();
  if (d->b == 0) return CONVFWD_OK;
  a.b = d->b; a.t = d->t; a.c = d->c; a.k = d->k; a.act = d->act; a.dtype = d->dtype;
  a.w = w; a.bias = bias; a.state = state; a.starts = (const uint8_t*)starts;
  a.y = y; a.state_out = state_out;
  return launched(launch_conv_fwd(a, (hipStream_t)stream));
}

int64_t convseq_conv_bwd_workspace(const convseq_conv_desc* d) {
  const int rc = check_conv(d);
  return rc < 0 ? rc : conv_bwd_work_bytes(d->b, d->t, d->c, d->k);
}

int convseq_conv_bwd(const convseq_conv_desc* d, const convseq_rows* dy, const convseq_rows* x,
                     const convseq_kept* kept, const void* w, const void* bias, const void* state,
                     const void* starts, const void* dstate_out, void* dx, void* dw, void* dbias, void* dstate,
                     void* workspace, void* stream) {
  const int rc = check_conv(d);
  if (rc < 0) return rc;
  if (!x == !kept) return x ? CONVFWD_ERR_BAD_DESC : CONVFWD_ERR_NULL;
  const int eb = elem_bytes(d->dtype);
  const int64_t n = (int64_t)d->b * d->t * d->c, rows = (int64_t)d->b * (d->k - 1) * d->c;
  ConvArgs a{};
  Buffers buf;
  buf.rows(dy, d->b, d->t, d->c, eb, &a.dy);
  if (x) buf.rows(x, d->b, d->t, d->c, eb, &a.x);
  buf.kept(kept, d->b, d->t, d->c, false, &a.kept);
  buf.in(w, (int64_t)d->c * d->k * eb, eb);
  buf.in(bias, (int64_t)d->c * eb, eb, false);
  buf.in(state, rows * eb, eb, false);
  buf.in(starts, (int64_t)d->b * d->t, 1, false);
  buf.in(dstate_out, rows * eb, eb, false);
  buf.out(dx, n * eb, eb);
  buf.out(dw, (int64_t)d->c * d->k * 4, 4);
  buf.out(dbias, (int64_t)d->c * 4, 4, false);
  buf.out(dstate, rows * eb, eb, false);
  buf.out(workspace, conv_bwd_work_bytes(d->b, d->t, d->c, d->k), 16);
  if (buf.result() < 0) return buf.result();
  a.b = d->b; a.t = d->t; a.c = d->c; a.k = d->k; a.act = d->act; a.dtype = d->dtype;
  a.w = w; a.bias = bias; a.state = state; a.starts = (const uint8_t*)starts;
  a.dstate_out = dstate_out; a.dx = dx; a.dw = (float*)dw; a.dbias = (float*)dbias; a.dstate = dstate;
  a.work = (float*)workspace;
  const auto launch = d->dtype == CONVFWD_F32   ? launch_conv_bwd_f32
                      : d->dtype == CONVFWD_F16 ? launch_conv_bwd_f16
                                                : launch_conv_bwd_bf16;
  return launched(launch(a, (hipStream_t)stream));
}

int convseq_conv_step(const convseq_conv_desc* d, const void* x, int64_t x_row, const void* w,
                      const void* bias, const void* state, void* state_out, const void* slots, int32_t n_slots,
                      void* y, void* stream) {
  if (!d) return CONVFWD_ERR_NULL;
  convseq_conv_desc one = *d;
  one.t = 1;
  const int rc = check_conv(&one);
  if (rc < 0) return rc;
  if (n_slots < 0 || (!slots && n_slots < d->b)) return CONVFWD_ERR_BAD_DESC;
  const int eb = elem_bytes(d->dtype);
  const int64_t rows = (int64_t)n_slots * (d->k - 1) * d->c * eb;
  ConvStepArgs a{};
  Buffers buf;
  const convseq_rows xr = {x, x_row, 0};
  Rows view;
  buf.rows(&xr, d->b, 1, d->c, eb, &view);
  buf.in(w, (int64_t)d->c * d->k * eb, eb);
  buf.in(bias, (int64_t)d->c * eb, eb, false);
  buf.in(slots, (int64_t)d->b * 4, 4, false);
  buf.out(y, (int64_t)d->b * d->c * eb, eb);
  if (state != state_out) buf.in(state, rows, eb);
  buf.out(state_out, rows, eb);
  if (buf.result() < 0) return buf.result();
  if (d->b == 0) return CONVFWD_OK;
  a.b = d->b; a.c = d->c; a.k = d->k; a.act = d->act; a.dtype = d->dtype; a.n_slots = n_slots;
  a.x = x; a.x_row = x_row; a.w = w; a.bias = bias; a.state = state; a.state_out = state_out;
  a.slots = (const int32_t*)slots; a.y = y;
  return launched(launch_conv_step(a, (hipStream_t)stream));
}

int64_t convseq_scan_fwd_workspace(const convseq_scan_desc* d) {
  const int rc = check_scan(d);
  return rc < 0 ? rc : scan_fwd_work_bytes(d->b, d->t, d->c);
}

int64_t convseq_scan_bwd_workspace(const convseq_scan_desc* d) {
  const int rc = check_scan(d);
  return rc < 0 ? rc : scan_bwd_work_bytes(d->b, d->t, d->c);
}

int convseq_scan_fwd(const convseq_scan_desc* d, const convseq_rows* x, const convseq_rows* gate_r,
                     const convseq_rows* gate_i, const void* lam, const void* h0, const void* starts, void* y,
                     void* h_last, void* states, const convseq_kept kept[3], void* workspace, void* stream) {
  const int rc = check_scan(d);
  if (rc < 0) return rc;
  const int eb = elem_bytes(d->dtype);
  const int64_t n = (int64_t)d->b * d->t * d->c, bc = (int64_t)d->b * d->c;
  const int64_t pieces = ((int64_t)d->t + kEvery - 1) / kEvery;
  ScanArgs a{};
  Buffers buf;
  buf.rows(x, d->b, d->t, d->c, eb, &a.x);
  buf.rows(gate_r, d->b, d->t, d->c, eb, &a.r);
  buf.rows(gate_i, d->b, d->t, d->c, eb, &a.i);
  buf.in(lam, (int64_t)d->c * 4, 4);
  buf.in(h0, bc * 4, 4, false);
  buf.in(starts, (int64_t)d->b * d->t, 1, false);
  buf.out(y, n * eb, eb);
  buf.out(h_last, bc * 4, 4, false);
  buf.out(states, bc * pieces * 4, 4, false);
  for (int k = 0; kept && k < 3; ++k) buf.kept(kept + k, d->b, d->t, d->c, true, &a.kept[k]);
  buf.out(workspace, scan_fwd_work_bytes(d->b, d->t, d->c), 16);
  if (buf.result() < 0) return buf.result();
  if (d->b == 0) return CONVFWD_OK;
  a.b = d->b; a.t = d->t; a.c = d->c; a.dtype = d->dtype; a.decay = d->decay;
  a.lam = (const float*)lam; a.h0 = (const float*)h0; a.starts = (const uint8_t*)starts;
  a.y = y; a.h_last = (float*)h_last; a.states = (float*)states; a.work = workspace;
  return launched(launch_scan_fwd(a, (hipStream_t)stream));
}

int convseq_scan_bwd(const convseq_scan_desc* d, const convseq_rows* dy, const convseq_rows* x,
                     const convseq_rows* gate_r, const convseq_rows* gate_i, const convseq_kept kept[3],
                     const void* lam, const void* states, const void* starts, const void* dh_last, void* dx,
                     void* dgate_r, void* dgate_i, void* dlam, void* dh0, void* workspace, void* stream) {
  const int rc = check_scan(d);
  if (rc < 0) return rc;
  const bool plain = x || gate_r || gate_i;
  if (plain && kept) return CONVFWD_ERR_BAD_DESC;
  if (!kept && !(x && gate_r && gate_i)) return CONVFWD_ERR_NULL;
  const int eb = elem_bytes(d->dtype);
  const int64_t n = (int64_t)d->b * d->t * d->c, bc = (int64_t)d->b * d->c;
  const int64_t pieces = ((int64_t)d->t + kEvery - 1) / kEvery;
  ScanArgs a{};
  Buffers buf;
  buf.rows(dy, d->b, d->t, d->c, eb, &a.dy);
  if (kept) {
    for (int k = 0; k < 3; ++k) buf.kept(kept + k, d->b, d->t, d->c, false, &a.kept[k]);
  } else {
    buf.rows(x, d->b, d->t, d->c, eb, &a.x);
    buf.rows(gate_r, d->b, d->t, d->c, eb, &a.r);
    buf.rows(gate_i, d->b, d->t, d->c, eb, &a.i);
  }
  buf.in(lam, (int64_t)d->c * 4, 4);
  buf.in(states, bc * pieces * 4, 4);
  buf.in(starts, (int64_t)d->b * d->t, 1, false);
  buf.in(dh_last, bc * 4, 4, false);
  buf.out(dx, n * eb, eb);
  buf.out(dgate_r, n * eb, eb);
  buf.out(dgate_i, n * eb, eb);
  buf.out(dlam, (int64_t)d->c * 4, 4);
  buf.out(dh0, bc * 4, 4, false);
  buf.out(workspace, scan_bwd_work_bytes(d->b, d->t, d->c), 16);
  if (buf.result() < 0) return buf.result();
  a.b = d->b; a.t = d->t; a.c = d->c; a.dtype = d->dtype; a.decay = d->decay;
  a.lam = (const float*)lam; a.states_in = (const float*)states; a.starts = (const uint8_t*)starts;
  a.dh_last = (const float*)dh_last; a.dx = dx; a.dr = dgate_r; a.di = dgate_i;
  a.dlam = (float*)dlam; a.dh0 = (float*)dh0; a.work = workspace;
  return launched(launch_scan_bwd(a, (hipStream_t)stream));
}

int convseq_scan_step(const convseq_scan_desc* d, const void* x, int64_t x_row, const void* gate_r,
                      int64_t r_row, const void* gate_i, int64_t i_row, const void* lam, const void* state,
                      void* state_out, const void* slots, int32_t n_slots, void* y, void* stream) {
  if (!d) return CONVFWD_ERR_NULL;
  convseq_scan_desc one = *d;
  one.t = 1;
  const int rc = check_scan(&one);
  if (rc < 0) return rc;
  if (n_slots < 0 || (!slots && n_slots < d->b)) return CONVFWD_ERR_BAD_DESC;
  const int eb = elem_bytes(d->dtype);
  const int64_t rows = (int64_t)n_slots * d->c * 4;
  ScanStepArgs a{};
  Buffers buf;
  const convseq_rows in[3] = {{x, x_row, 0}, {gate_r, r_row, 0}, {gate_i, i_row, 0}};
  for (int k = 0; k < 3; ++k) {
    Rows view;
    buf.rows(in + k, d->b, 1, d->c, eb, &view);
  }
  buf.in(lam, (int64_t)d->c * 4, 4);
  buf.in(slots, (int64_t)d->b * 4, 4, false);
  buf.out(y, (int64_t)d->b * d->c * eb, eb);
  if (state != state_out) buf.in(state, rows, 4);
  buf.out(state_out, rows, 4);
  if (buf.result() < 0) return buf.result();
  if (d->b == 0) return CONVFWD_OK;
  a.b = d->b; a.c = d->c; a.dtype = d->dtype; a.decay = d->decay; a.n_slots = n_slots;
  a.x = x; a.r = gate_r; a.i = gate_i; a.x_row = x_row; a.r_row = r_row; a.i_row = i_row;
  a.lam = (const float*)lam; a.state = (const float*)state; a.state_out = (float*)state_out;
  a.slots = (const int32_t*)slots; a.y = y;
  return launched(launch_scan_step(a, (hipStream_t)stream));
}

int convseq_pack8(int32_t b, int32_t t, int32_t c, int32_t dtype, const convseq_rows* x,
                  const convseq_kept* kept, void* stream) {
  const int rc = check_extents(b, t, c, dtype);
  if (rc < 0) return rc;
  if (!kept) return CONVFWD_ERR_NULL;
  Buffers buf;
  Rows rows;
  Kept k;
  buf.rows(x, b, t, c, elem_bytes(dtype), &rows);
  buf.kept(kept, b, t, c, true, &k);
  if (buf.result() < 0) return buf.result();
  if (b == 0 || t == 0) return CONVFWD_OK;
  return launched(launch_pack8(b, t, c, dtype, rows, k, (hipStream_t)stream));
}

int convseq_unpack8(int32_t b, int32_t t, int32_t c, int32_t dtype, const convseq_kept* kept, void* out,
                    void* stream) {
  const int rc = check_extents(b, t, c, dtype);
  if (rc < 0) return rc;
  if (!kept) return CONVFWD_ERR_NULL;
  Buffers buf;
  Kept k;
  const int eb = elem_bytes(dtype);
  buf.kept(kept, b, t, c, false, &k);
  buf.out(out, (int64_t)b * t * c * eb, eb);
  if (buf.result() < 0) return buf.result();
  if (b == 0 || t == 0) return CONVFWD_OK;
  return launched(launch_unpack8(b, t, c, dtype, k, out, (hipStream_t)stream));
}

}  // extern "C"
