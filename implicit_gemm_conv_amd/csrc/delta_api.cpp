// delta_api.cpp -- the C ABI declared in include/convdelta.h: validation, the
// workspace's layout and the launches on the caller's stream.  No device memory is
// allocated here and nothing is synchronised.
#include "../../include/convdelta.h"

#include <math.h>

#include "conv_params.h"
#include "delta_params.h"
#include "seq_buffers.h"

using namespace convdelta;
using convseq::Buffers;
using convseq::elem_bytes;
using convseq::launched;

namespace {

int check(const convdelta_desc* d) {
  if (!d) return CONVFWD_ERR_NULL;
  if (d->b < 0 || d->t < 0 || d->hk < 1 || d->hv < 1 || d->dk < 1 || d->dv < 1) return CONVFWD_ERR_BAD_DESC;
  if (d->hv % d->hk || !isfinite(d->scale)) return CONVFWD_ERR_BAD_DESC;
  if (d->dtype != CONVFWD_F32 && d->dtype != CONVFWD_F16 && d->dtype != CONVFWD_BF16) return CONVFWD_ERR_UNSUPPORTED;
  if (d->dk > CONVDELTA_MAX_DK) return CONVFWD_ERR_UNSUPPORTED;
  // workgroups of up to 512 threads: one for each value head and 16 columns (rounded up to 32), where the heads are
  // rounded up to 8, or for each chunk and value head; a grid holds less than 2^32 threads
  const int64_t lim = (int64_t)1 << 23, chunks = ((int64_t)d->t + kChunk - 1) / kChunk, blocks = ((int64_t)d->dv + 31) / 32 * 2;
  const int64_t heads = ((int64_t)d->b * d->hv + 7) / 8 * 8;
  if (d->t >= 1 << 30 || d->hv >= lim || blocks >= lim || heads >= lim || heads * blocks >= lim) return CONVFWD_ERR_TOO_LARGE;
  if (chunks * heads >= lim) return CONVFWD_ERR_TOO_LARGE;
  // offsets of 32 bits: 64 rows of v or y, 128 rows of a state
  if ((int64_t)d->hv * d->dv >= (int64_t)1 << 23 || d->dv >= 1 << 22) return CONVFWD_ERR_TOO_LARGE;
  // ... and one for each 2048 elements of q and k
  if (d->hk * (int64_t)d->b >= lim || d->hk * (int64_t)d->b * chunks * 4 >= lim) return CONVFWD_ERR_TOO_LARGE;
  return CONVFWD_OK;
}

int64_t chunks_of(const convdelta_desc* d) { return ((int64_t)d->t + kChunk - 1) / kChunk; }

int dkp_of(const convdelta_desc* d) { return (d->dk + 7) / 8 * 8; }

// Lays the workspace out from `base` and returns its bytes.
int64_t lay_out(const convdelta_desc* d, bool backward, char* base, Work* w) {
  const int64_t n = (int64_t)d->b * d->hv * chunks_of(d), dvp = ((int64_t)d->dv + 31) / 32 * 32;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    char* p = base ? base + at : nullptr;
    at += (n * bytes + 15) / 16 * 16;
    return p;
  };
  *w = Work{};
  if (!backward) {
    w->solve = take(kMatrix);
    w->read = take(kMatrix);
  } else {
    w->solve_t = take(kMatrix);
    w->read_t = take(kMatrix);
    w->sums = (double*)take(8 * kChunk);
    w->seq = (int*)take(4 * kChunk);
    w->z = (float*)take(4 * kChunk * dvp);
    w->dstate = (float*)take(4 * d->dk * dvp);
  }
  w->rows = (float*)take(4 * 4 * kChunk);
  for (void** copy : {&w->q, &w->k}) {
    *copy = base ? base + at : nullptr;
    at += (int64_t)d->b * d->t * d->hk * dkp_of(d) * elem_bytes(d->dtype);  // whole 16 bytes a row
  }
  return at;
}

int64_t work_bytes(const convdelta_desc* d, bool backward) {
  const int rc = check(d);
  Work w;
  return rc < 0 ? rc : lay_out(d, backward, nullptr, &w);
}

// A (B, T, H, D) view; the step calls pass t = 1.
void heads(Buffers* buf, const convdelta_heads* x, int64_t b, int64_t t, int64_t h, int64_t d, int elem, Heads* to) {
  *to = Heads{nullptr, 0, 0, 0};
  const convseq_rows bad = {nullptr, -1, -1}, far = {nullptr, (int64_t)1 << 62, 0};
  convseq::Rows unused;
  if (!x) return buf->rows(nullptr, 1, 1, 1, elem, &unused);
  if (x->batch_stride < 0 || x->row_stride < 0 || x->head_stride < 0) return buf->rows(&bad, 1, 1, 1, elem, &unused);
  const int64_t n[3] = {b > 1 ? b - 1 : 0, t > 1 ? t - 1 : 0, h - 1};
  const int64_t s[3] = {x->batch_stride, x->row_stride, x->head_stride};
  int64_t last = d;
  for (int i = 0; i < 3; ++i) {
    // 2^60 bytes each is past any address range; keeps the sum in 64 bits
    if (n[i] && s[i] > ((int64_t)1 << 58) / n[i]) return buf->rows(&far, 3, 1, 1, elem, &unused);
    last += n[i] * s[i];
  }
  buf->in(x->data, b == 0 || t == 0 ? 0 : last * elem, elem);
  *to = Heads{x->data, x->batch_stride, x->row_stride, x->head_stride};
}

// 64 rows of at most 2^22 elements have offsets of 32 bits.
bool near_rows(const Heads& h) { return h.st < (int64_t)1 << 23; }

// Rows of d elements are whole pieces of 8, 16-byte aligned.
bool pieces(const Heads& h, int d, int elem) {
  return d % 8 == 0 && near_rows(h) && ((uintptr_t)h.p | (uint64_t)(h.sb * elem) | (uint64_t)(h.st * elem) | (uint64_t)(h.sh * elem)) % 16 == 0;
}

void fill(DeltaArgs* a, const convdelta_desc* d) {
  a->b = d->b; a->t = d->t; a->hk = d->hk; a->hv = d->hv; a->dk = d->dk; a->dv = d->dv; a->dtype = d->dtype;
  a->chunks = (int)chunks_of(d);
  a->dvp = (d->dv + 31) / 32 * 32;
  a->dkp = dkp_of(d);
  a->scale = d->scale;
}

// What is launched before the recurrence; q and k become aligned rows.
int prepare(DeltaArgs* a, bool backward, hipStream_t s) {
  const int eb = elem_bytes(a->dtype);
  if (!pieces(a->q, a->dk, eb) || !pieces(a->k, a->dk, eb)) {
    const int rc = launched(launch_delta_pack(*a, a->q, a->k, s));
    if (rc < 0) return rc;
    a->q = packed_rows(a->w.q, a->t, a->hk, a->dkp);
    a->k = packed_rows(a->w.k, a->t, a->hk, a->dkp);
  }
  return launched(launch_delta_prep(*a, backward, s));
}

typedef hipError_t (*Launch)(const DeltaArgs&, hipStream_t);

}  // namespace

extern "C" {

int64_t convdelta_fwd_workspace(const convdelta_desc* d) { return work_bytes(d, false); }
int64_t convdelta_bwd_workspace(const convdelta_desc* d) { return work_bytes(d, true); }

int convdelta_fwd(const convdelta_desc* d, const convdelta_heads* q, const convdelta_heads* k,
                  const convdelta_heads* v, const void* log_decay, const void* beta, const void* h0,
                  const void* starts, void* y, void* h_last, void* states, void* x, void* workspace, void* stream) {
  const int64_t work = work_bytes(d, false);
  if (work < 0) return (int)work;
  const int eb = elem_bytes(d->dtype);
  if (!states != !x && d->b > 0 && d->t > 0) return CONVFWD_ERR_NULL;
  const int64_t rows = (int64_t)d->b * d->t, size = (int64_t)d->b * d->hv * d->dk * d->dv * 4;
  DeltaArgs a{};
  Buffers buf;
  heads(&buf, q, d->b, d->t, d->hk, d->dk, eb, &a.q);
  heads(&buf, k, d->b, d->t, d->hk, d->dk, eb, &a.k);
  heads(&buf, v, d->b, d->t, d->hv, d->dv, eb, &a.v);
  buf.in(log_decay, rows * d->hv * 4, 4);
  buf.in(beta, rows * d->hv * 4, 4);
  buf.in(h0, size, 4, false);
  buf.in(starts, rows, 1, false);
  buf.out(y, rows * d->hv * d->dv * eb, eb);
  buf.out(h_last, size, 4);
  buf.out(states, size * chunks_of(d), 4, false);
  buf.out(x, rows * d->hv * d->dv * 4, 4, false);
  buf.out(workspace, work, 16);
  if (buf.result() < 0) return buf.result();
  if (!near_rows(a.v)) return CONVFWD_ERR_TOO_LARGE;
  if (d->b == 0) return CONVFWD_OK;
  fill(&a, d);
  a.log_decay = (const float*)log_decay; a.beta = (const float*)beta; a.h0 = (const float*)h0;
  a.starts = (const uint8_t*)starts; a.y = y; a.h_last = (float*)h_last; a.states = (float*)states;
  a.x = (float*)x;
  lay_out(d, false, (char*)workspace, &a.w);
  const hipStream_t s = (hipStream_t)stream;
  if (a.chunks > 0) {
    const int rc = prepare(&a, false, s);
    if (rc < 0) return rc;
  }
  static const Launch fwd[3] = {launch_delta_fwd_f32, launch_delta_fwd_f16, launch_delta_fwd_bf16};
  return launched(fwd[d->dtype](a, s));
}

int convdelta_bwd(const convdelta_desc* d, const convdelta_heads* dy, const convdelta_heads* q,
                  const convdelta_heads* k, const convdelta_heads* v, const void* log_decay, const void* beta,
                  const void* states, const void* x, const void* starts, const void* dh_last, void* dq, void* dk,
                  void* dv, void* dlog_decay, void* dbeta, void* dh0, void* workspace, void* stream) {
  const int64_t work = work_bytes(d, true);
  if (work < 0) return (int)work;
  const int eb = elem_bytes(d->dtype);
  const int64_t rows = (int64_t)d->b * d->t, size = (int64_t)d->b * d->hv * d->dk * d->dv * 4;
  DeltaArgs a{};
  Buffers buf;
  heads(&buf, dy, d->b, d->t, d->hv, d->dv, eb, &a.dy);
  heads(&buf, q, d->b, d->t, d->hk, d->dk, eb, &a.q);
  heads(&buf, k, d->b, d->t, d->hk, d->dk, eb, &a.k);
  heads(&buf, v, d->b, d->t, d->hv, d->dv, eb, &a.v);
  buf.in(log_decay, rows * d->hv * 4, 4);
  buf.in(beta, rows * d->hv * 4, 4);
  buf.in(states, size * chunks_of(d), 4);
  buf.in(x, rows * d->hv * d->dv * 4, 4);
  buf.in(starts, rows, 1, false);
  buf.in(dh_last, size, 4, false);
  buf.out(dq, rows * d->hk * d->dk * eb, eb);
  buf.out(dk, rows * d->hk * d->dk * eb, eb);
  buf.out(dv, rows * d->hv * d->dv * eb, eb);
  buf.out(dlog_decay, rows * d->hv * 4, 4);
  buf.out(dbeta, rows * d->hv * 4, 4);
  buf.out(dh0, size, 4);
  buf.out(workspace, work, 16);
  if (buf.result() < 0) return buf.result();
  if (!near_rows(a.v) || !near_rows(a.dy)) return CONVFWD_ERR_TOO_LARGE;
  if (d->b == 0) return CONVFWD_OK;
  fill(&a, d);
  a.log_decay = (const float*)log_decay; a.beta = (const float*)beta; a.states_in = (const float*)states;
  a.x_in = (const float*)x;
  a.starts = (const uint8_t*)starts; a.dh_last = (const float*)dh_last;
  a.dq = dq; a.dk_ = dk; a.dv_ = dv; a.dlog_decay = (float*)dlog_decay; a.dbeta = (float*)dbeta; a.dh0 = (float*)dh0;
  a.whole = pieces(a.dy, d->dv, eb);
  lay_out(d, true, (char*)workspace, &a.w);
  const hipStream_t s = (hipStream_t)stream;
  static const Launch bwd[3] = {launch_delta_bwd_f32, launch_delta_bwd_f16, launch_delta_bwd_bf16};
  static const Launch grad[3] = {launch_delta_grad_f32, launch_delta_grad_f16, launch_delta_grad_bf16};
  int rc = CONVFWD_OK;
  if (a.chunks > 0) rc = prepare(&a, true, s);
  if (rc == CONVFWD_OK) rc = launched(bwd[d->dtype](a, s));
  if (a.chunks > 0 && rc == CONVFWD_OK) rc = launched(grad[d->dtype](a, s));
  return rc;
}

int convdelta_step(const convdelta_desc* d, const convdelta_heads* q, const convdelta_heads* k,
                   const convdelta_heads* v, const void* log_decay, const void* beta, const void* state,
                   void* state_out, const void* slots, int32_t n_slots, void* y, void* stream) {
  if (!d) return CONVFWD_ERR_NULL;
  convdelta_desc one = *d;
  one.t = 1;
  const int rc = check(&one);
  if (rc < 0) return rc;
  if (n_slots < 0 || (!slots && n_slots < d->b)) return CONVFWD_ERR_BAD_DESC;
  const int eb = elem_bytes(d->dtype);
  const int64_t gates = (int64_t)d->b * d->hv * 4, each = (int64_t)d->hv * d->dk * d->dv * 4;
  if (n_slots && each > ((int64_t)1 << 60) / n_slots) return CONVFWD_ERR_TOO_LARGE;
  DeltaStepArgs a{};
  Buffers buf;
  heads(&buf, q, d->b, 1, d->hk, d->dk, eb, &a.q);
  heads(&buf, k, d->b, 1, d->hk, d->dk, eb, &a.k);
  heads(&buf, v, d->b, 1, d->hv, d->dv, eb, &a.v);
  buf.in(log_decay, gates, 4);
  buf.in(beta, gates, 4);
  buf.in(slots, (int64_t)d->b * 4, 4, false);
  buf.out(y, (int64_t)d->b * d->hv * d->dv * eb, eb);
  if (state != state_out) buf.in(state, each * n_slots, 4);
  buf.out(state_out, each * n_slots, 4);
  if (buf.result() < 0) return buf.result();
  if (d->b == 0) return CONVFWD_OK;
  a.b = d->b; a.hk = d->hk; a.hv = d->hv; a.dk = d->dk; a.dv = d->dv; a.dtype = d->dtype; a.n_slots = n_slots;
  a.scale = d->scale; a.log_decay = (const float*)log_decay; a.beta = (const float*)beta;
  a.state = (const float*)state; a.state_out = (float*)state_out; a.slots = (const int32_t*)slots; a.y = y;
  return launched(launch_delta_step(a, (hipStream_t)stream));
}

}  // extern "C"
