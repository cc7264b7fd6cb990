// norm_api.cpp -- the C ABI declared in include/convnorm.h: validation, the cut
// of the problem and the launches on the caller's stream.  No device memory is
// allocated here and nothing is synchronised.
#include "../../include/convnorm.h"

#include <algorithm>

#include "norm_params.h"
#include "seq_buffers.h"

namespace convnorm {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

}  // namespace

// `whole_pieces`: every row of the inputs and outputs is 16-byte aligned.
Plan make_plan(int n, int p, int c, int groups, int elem, bool whole_pieces, bool backward) {
  Plan pl{};
  const int cg = c / groups, wide = 16 / elem, held = p >= kFewRows ? 1 : backward ? kTeamHeldBwd : kTeamHeld;
  // ---- a team for each (n, group) ----
  // Up to 256 pieces a lane holds one (8 positions of 1024 channels in 8 groups, n 4096, bf16, forward and backward: 41 and
  // 59 us, in tiles 60 and 99; one position of 8192 in 4 groups, n 16384: 147 and 186 us, in tiles 684 and 1398).  More
  // pieces a lane are faster than tiles only where these would be of few rows (one position of 4096 channels in one group,
  // n 4096: 59 and 64 us, in tiles 92 and 158; 4 positions of 2048, n 2048: 55 and 70, in tiles 39 and 67).
  const int v = whole_pieces && cg % wide == 0 ? wide : 1;
  const int64_t pieces = (int64_t)p * (cg / v);
  if (pieces <= (int64_t)kThreads * held) {
    pl.v = v;
    pl.team = 1;
    while (pl.team < pieces && pl.team < kThreads) pl.team *= 2;
    pl.held = (int)std::max<int64_t>(1, ceil_div(pieces, pl.team));
    const int teams = kThreads / pl.team;
    // as many lanes as the chip holds at once, each walking over n with its channels' parameters in registers (16384 rows
    // of 16 groups of 128, bf16: forward 43 us with 2048 workgroups, 44 and 49 us with half and twice as many and 125 us
    // with a team for each (n, group); backward, with the columns, 61 us with 1024, 67 us with 512)
    pl.step = std::min<int64_t>(n, std::max<int64_t>(1, (int64_t)(backward ? 1024 : 2048) * teams / groups));
    pl.blocks = ceil_div(pl.step * groups, teams);
    pl.rows = pl.step * p;
    return pl;
  }
  // ---- tiles of positions ----
  // pieces of 16 bytes where a workgroup's channels can be whole groups and whole pieces
  pl.v = 1;
  int unit = cg;  // the fewest channels that are both
  if (whole_pieces && c % wide == 0) {
    const int u = wide / gcd(wide, cg) * cg;
    if (cg % wide == 0 || u <= kThreads * wide) {
      pl.v = wide;
      unit = u;
    }
  }
  const int most = kThreads * pl.v;
  if (cg > most) {
    pl.slices = (int)ceil_div(cg, most);
    pl.cw = most;
    pl.k = 1;
    pl.cblocks = groups * pl.slices;
  } else {
    pl.slices = 1;
    pl.k = std::min(most / unit * (unit / cg), groups);
    pl.cw = pl.k * cg;
    pl.cblocks = (int)ceil_div(groups, pl.k);
  }
  const int rw = kThreads / (pl.cw / pl.v), least = rw * 8;
  // eight workgroups a compute unit, of at least eight rows a thread
  const int64_t want = std::max<int64_t>(1, 2048 / ((int64_t)std::max(n, 1) * pl.cblocks));
  pl.per = (int)(ceil_div(std::max<int64_t>(ceil_div(p, want), least), rw * 4) * (rw * 4));
  pl.tiles = (int)ceil_div(p, pl.per);
  pl.blocks = (int64_t)n * pl.tiles * pl.cblocks;
  pl.rows = (int64_t)n * pl.tiles;
  // Every workgroup of the second pass joins the sums of its own groups where a thread has few of them, for a launch
  // less (1 group of 64^3 x 64, fp16: both passes 65 us for 79); else that is left to a launch between the passes
  // (32^3 x 128 in 32 groups: the second pass took 31 us for 12).
  pl.joint = (int64_t)pl.slices * pl.tiles > (int64_t)kJoinEach * join_lanes(pl.slices == 1 ? pl.k : 1);
  return pl;
}

namespace {

int64_t part_bytes(const Plan& pl, int n, int groups) {
  return pl.team ? 0 : ceil_div((int64_t)n * groups * pl.slices * pl.tiles * 8, 16) * 16;
}

int64_t two_bytes(const Plan& pl, int n, int groups) { return pl.joint ? ceil_div((int64_t)n * groups * 8, 16) * 16 : 0; }

}  // namespace

int64_t fwd_work_bytes(const Plan& pl, int n, int groups) { return part_bytes(pl, n, groups); }
int64_t bwd_work_bytes(const Plan& pl, int n, int c, int groups) {
  return part_bytes(pl, n, groups) + two_bytes(pl, n, groups) + pl.rows * c * 8;
}

}  // namespace convnorm

using namespace convnorm;
using convseq::Buffers;
using convseq::elem_bytes;
using convseq::launched;

namespace {

int check(const convnorm_desc* d) {
  if (!d) return CONVFWD_ERR_NULL;
  if (d->n < 0 || d->p < 0 || d->c < 1 || d->groups < 1 || d->act < 0 || d->act > CONVSEQ_ACT_SILU) return CONVFWD_ERR_BAD_DESC;
  if (d->c % d->groups || !(d->eps >= 0.f && d->eps < 1e30f)) return CONVFWD_ERR_BAD_DESC;
  if (d->dtype != CONVFWD_F32 && d->dtype != CONVFWD_F16 && d->dtype != CONVFWD_BF16) return CONVFWD_ERR_UNSUPPORTED;
  if (d->param_dtype != d->dtype && d->param_dtype != CONVFWD_F32) return CONVFWD_ERR_UNSUPPORTED;
  // channels of a row and positions of an n in 32 bits with room for a tile; the grids' threads in 32 bits
  if (d->c >= 1 << 26 || d->p >= 1 << 30 || (int64_t)d->n * d->groups >= (int64_t)1 << 30) return CONVFWD_ERR_TOO_LARGE;
  if ((int64_t)d->n * d->p >= ((int64_t)1 << 56) / d->c) return CONVFWD_ERR_TOO_LARGE;
  return CONVFWD_OK;
}

int check_plan(const Plan& pl, const convnorm_desc* d) {
  const int64_t lim = (int64_t)1 << 24;  // workgroups of 256 threads
  if (pl.blocks >= lim || (!pl.team && std::max(pl.blocks, (int64_t)d->n * d->groups) + d->c >= lim)) return CONVFWD_ERR_TOO_LARGE;
  return CONVFWD_OK;
}

// The plan whose workspace is largest, whatever the buffers' alignment turns out to be.
int64_t work_bytes(const convnorm_desc* d, bool backward) {
  const int rc = check(d);
  if (rc < 0) return rc;
  int64_t most = 0;
  for (const bool whole : {false, true}) {
    const Plan pl = make_plan(d->n, d->p, d->c, d->groups, elem_bytes(d->dtype), whole, backward);
    if (check_plan(pl, d) < 0) return CONVFWD_ERR_TOO_LARGE;
    most = std::max(most, backward ? bwd_work_bytes(pl, d->n, d->c, d->groups) : fwd_work_bytes(pl, d->n, d->groups));
  }
  return most;
}

void fill(NormArgs* a, const convnorm_desc* d) {
  a->n = d->n; a->p = d->p; a->c = d->c; a->groups = d->groups; a->act = d->act; a->dtype = d->dtype;
  a->param_f32 = d->param_dtype == CONVFWD_F32;
  a->eps = d->eps;
}

bool aligned(const void* p) { return (uintptr_t)p % 16 == 0; }

}  // namespace

extern "C" {

int64_t convnorm_group_fwd_workspace(const convnorm_desc* d) { return work_bytes(d, false); }
int64_t convnorm_group_bwd_workspace(const convnorm_desc* d) { return work_bytes(d, true); }

int convnorm_group_fwd(const convnorm_desc* d, const convseq_rows* x, const void* weight, const void* bias, void* y,
                       void* mean, void* rstd, void* workspace, void* stream) {
  const int64_t work = work_bytes(d, false);
  if (work < 0) return (int)work;
  const int eb = elem_bytes(d->dtype), pb = elem_bytes(d->param_dtype);
  const int64_t stats = (int64_t)d->n * d->groups * 4;
  NormArgs a{};
  Buffers buf;
  buf.rows(x, d->n, d->p, d->c, eb, &a.x);
  buf.in(weight, (int64_t)d->c * pb, pb, false);
  buf.in(bias, (int64_t)d->c * pb, pb, false);
  buf.out(y, (int64_t)d->n * d->p * d->c * eb, eb);
  buf.out(mean, stats, 4);
  buf.out(rstd, stats, 4);
  buf.out(workspace, work, 16);
  if (buf.result() < 0) return buf.result();
  if (d->n == 0) return CONVFWD_OK;
  fill(&a, d);
  a.weight = weight; a.bias = bias; a.y = y; a.mean = (float*)mean; a.rstd = (float*)rstd; a.part = (float*)workspace;
  const bool whole = (int64_t)d->c * eb % 16 == 0 && aligned(y) && convseq::pieces(a.x, 16, eb);
  a.plan = make_plan(d->n, d->p, d->c, d->groups, eb, whole, false);
  return launched(a.plan.team ? launch_norm_team_fwd(a, (hipStream_t)stream) : launch_norm_fwd(a, (hipStream_t)stream));
}

int convnorm_group_bwd(const convnorm_desc* d, const convseq_rows* dy, const convseq_rows* x, const void* weight,
                       const void* bias, const void* mean, const void* rstd, void* dx, void* dweight, void* dbias,
                       void* workspace, void* stream) {
  const int64_t work = work_bytes(d, true);
  if (work < 0) return (int)work;
  const int eb = elem_bytes(d->dtype), pb = elem_bytes(d->param_dtype);
  const int64_t stats = (int64_t)d->n * d->groups * 4;
  NormArgs a{};
  Buffers buf;
  buf.rows(dy, d->n, d->p, d->c, eb, &a.dy);
  buf.rows(x, d->n, d->p, d->c, eb, &a.x);
  buf.in(weight, (int64_t)d->c * pb, pb, false);
  buf.in(bias, (int64_t)d->c * pb, pb, false);
  buf.in(mean, stats, 4);
  buf.in(rstd, stats, 4);
  buf.out(dx, (int64_t)d->n * d->p * d->c * eb, eb);
  buf.out(dweight, (int64_t)d->c * 4, 4, false);
  buf.out(dbias, (int64_t)d->c * 4, 4, false);
  buf.out(workspace, work, 16);
  if (buf.result() < 0) return buf.result();
  fill(&a, d);
  a.weight = weight; a.bias = bias; a.mean_in = (const float*)mean; a.rstd_in = (const float*)rstd;
  a.y = dx; a.dweight = (float*)dweight; a.dbias = (float*)dbias;
  const hipStream_t s = (hipStream_t)stream;
  const bool params = dweight || dbias, whole = (int64_t)d->c * eb % 16 == 0 && aligned(dx) &&
                                                convseq::pieces(a.x, 16, eb) && convseq::pieces(a.dy, 16, eb);
  a.plan = make_plan(d->n, d->p, d->c, d->groups, eb, whole, true);
  if (d->n == 0 || d->p == 0) {
    a.plan.rows = 0;
    return params ? launched(launch_norm_columns(a, s)) : CONVFWD_OK;
  }
  char* w = (char*)workspace;
  a.part = (float*)w;
  w += part_bytes(a.plan, d->n, d->groups);
  a.two = (float*)w;
  w += two_bytes(a.plan, d->n, d->groups);
  a.chan = (float*)w;
  if (!a.plan.team) return launched(launch_norm_bwd(a, s));
  const int rc = launched(launch_norm_team_bwd(a, s));
  return rc < 0 || !params ? rc : launched(launch_norm_columns(a, s));
}

}  // extern "C"
