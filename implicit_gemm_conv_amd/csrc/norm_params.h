// norm_params.h -- plain parameter structs, the choice of a plan and launchers
// shared by the host side of include/convnorm.h (norm_api.cpp) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "seq_params.h"

namespace convnorm {

using convseq::Rows;

constexpr int kThreads = 256;
constexpr int kFewRows = 4;      // with fewer positions a lane may hold several pieces
constexpr int kTeamHeld = 4;     // pieces of 16 bytes (or values) of x that it then holds, forward
constexpr int kTeamHeldBwd = 2;  // backward, where it holds as many of dy and sums for the parameters

// How one problem is cut.
//   team > 0: each (n, group) belongs to a team of that many lanes, a power of two up to 256, which
//     holds it in registers; `v` channels a piece.
//   team = 0: workgroups of 256 threads own `cw` channels (whole groups, or a slice of one group where
//     a group has more) and `per` positions of one n: `tiles` of them along the positions, `cblocks`
//     along the channels, `slices` a group.
struct Plan {
  int v, team, held;
  int cw, k, cblocks, slices, per, tiles;
  int64_t blocks;  // of the team kernels
  int joint;       // tiles: a launch of its own joins their sums
  int64_t step;    // of the team kernels: they walk over n, this many in a turn
  int64_t rows;    // sums per channel that the backward pass leaves for the last step
};

struct NormArgs {
  int n, p, c, groups, act, dtype, param_f32;
  float eps;
  Plan plan;
  Rows x, dy;
  const void *weight, *bias;
  void* y;  // y or dx
  float *mean, *rstd;
  const float *mean_in, *rstd_in;
  float *dweight, *dbias;
  float* part;  // sums of tiles: (N, groups, slices, tiles) pairs
  float* two;   // backward, joint: the two means of each (n, group)
  float* chan;  // backward: sums per channel, (rows, C) pairs
};

// Threads of a workgroup that join the sums of one group, of its `groups`: a power of two of neighbouring ones, at most
// a wave, or all.
inline __host__ __device__ int join_lanes(int groups) {
  int of = kThreads;
  while (of > 1 && (of > kThreads / groups || (groups > 1 && of > 64))) of >>= 1;
  return of;
}
constexpr int kJoinEach = 8;  // sums that a thread joins at most where that is not a launch of its own

Plan make_plan(int n, int p, int c, int groups, int elem, bool whole_pieces, bool backward);
int64_t fwd_work_bytes(const Plan& pl, int n, int groups);
int64_t bwd_work_bytes(const Plan& pl, int n, int c, int groups);

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_team_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_team_bwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_columns(const NormArgs& a, hipStream_t s);  // dweight, dbias from `chan`

}  // namespace convnorm
