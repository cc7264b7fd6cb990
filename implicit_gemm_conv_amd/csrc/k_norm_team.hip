// k_norm_team.hip -- group norm where an (n, group) fits the registers of a
// team of lanes: rows normalised head by head, small images.  x is read once,
// the mean and the variance about it are taken from what is held.
#include "norm_device.h"

namespace convnorm {

namespace {

// Sum over a team of up to 256 lanes; with more than a wave, through LDS (every
// thread of the workgroup calls it the same number of times).
template <bool WIDE>
__device__ __forceinline__ float sum_of(float v, int team, float* lds) {
  if (!WIDE) return team_sum(v, team);
  v = team_sum(v, 64);
  const int wave = threadIdx.x / 64, of = team / 64;
  __syncthreads();  // what was read of the last sum
  if (threadIdx.x % 64 == 0) lds[wave] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < of; ++w) v += lds[wave / of * of + w];
  return v;
}

// Lane `lane` of a team holds pieces lane, lane + team, ... of its group; piece i is
// position i / (pieces a position), channels of piece i % (pieces a position).
template <typename T, int V, bool SILU, int H, bool WIDE>
__global__ __launch_bounds__(kThreads) void norm_team_fwd_kernel(NormArgs a) {
  __shared__ float lds[kThreads / 64];
  const int team = a.plan.team, lane = threadIdx.x % team;
  const int cg = a.c / a.groups, wide = cg / V, pieces = wide * a.p;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / team) + threadIdx.x / team;
  const int64_t n = item / a.groups;
  const int g = (int)(item % a.groups);
  const bool live = n < a.n;
  typedef Pack<T, V> P;
  float v[H][V];
  int ch[H];
  int64_t to[H];
  float sum = 0.f;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int i = lane + h * team;
    const int pos = i / wide;
    ch[h] = g * cg + i % wide * V;
    to[h] = live && i < pieces ? ((n * a.p + pos) * a.c + ch[h]) : -1;
    if (to[h] >= 0) {
      const P q = *(const P*)((const T*)a.x.p + n * a.x.sb + pos * a.x.st + ch[h]);
#pragma unroll
      for (int e = 0; e < V; ++e) sum += v[h][e] = q.get(e);
    }
  }
  const float inv = 1.f / (float)max(cg * a.p, 1);
  // about a first mean, whose own rounding the sum of the differences then takes out
  float mean = sum_of<WIDE>(sum, team, lds) * inv, off = 0.f;
  sum = 0.f;
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (to[h] >= 0)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        v[h][e] -= mean;
        off += v[h][e];
        sum = fmaf(v[h][e], v[h][e], sum);
      }
  off = sum_of<WIDE>(off, team, lds) * inv;
  mean += off;
  const float var = fmaf(-off, off, sum_of<WIDE>(sum, team, lds) * inv);
  const float rstd = 1.f / sqrtf(fmaxf(var, 0.f) + a.eps);
  if (live && lane == 0) {
    a.mean[item] = mean;
    a.rstd[item] = rstd;
  }
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (to[h] >= 0) {
      P q;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float w = param(a.weight, a.param_f32, a.dtype, ch[h] + e, 1.f);
        const float b = param(a.bias, a.param_f32, a.dtype, ch[h] + e, 0.f);
        q.set(e, activate<SILU>(fmaf((v[h][e] - off) * rstd, w, b)));
      }
      *(P*)((T*)a.y + to[h]) = q;
    }
}

// The same cut.  A team keeps its group of channels and walks over n, so that a
// lane's sums for the parameters stay in registers; they are left, a row for each
// position of each team, to the columns' kernel.
template <typename T, int V, bool SILU, int H, bool WIDE>
__global__ __launch_bounds__(kThreads) void norm_team_bwd_kernel(NormArgs a) {
  __shared__ float lds[kThreads / 64];
  const int team = a.plan.team, lane = threadIdx.x % team;
  const int cg = a.c / a.groups, wide = cg / V, pieces = wide * a.p;
  const int64_t id = (int64_t)blockIdx.x * (kThreads / team) + threadIdx.x / team;
  const int64_t rows = a.plan.rows / max(a.p, 1);  // teams of one group: n is walked in steps of it
  const int g = (int)(id % a.groups);
  const bool live = id < rows * a.groups;
  typedef Pack<T, V> P;
  float w[H][V], b[H][V], dw[H][V], db[H][V];
  int ch[H], pos[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int i = lane + h * team;
    pos[h] = i < pieces && live ? i / wide : -1;
    ch[h] = g * cg + i % wide * V;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[h][e] = b[h][e] = dw[h][e] = db[h][e] = 0.f;
      if (pos[h] >= 0) {
        w[h][e] = param(a.weight, a.param_f32, a.dtype, ch[h] + e, 1.f);
        b[h][e] = param(a.bias, a.param_f32, a.dtype, ch[h] + e, 0.f);
      }
    }
  }
  const float inv = 1.f / (float)max(cg * a.p, 1);
  // every team of a workgroup makes as many turns (the sums of wide teams wait for each other)
  const int64_t turns = (a.n + rows - 1) / rows;
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t n = id / a.groups + turn * rows;
    const bool here = live && n < a.n;
    const float mean = here ? a.mean_in[n * a.groups + g] : 0.f, rstd = here ? a.rstd_in[n * a.groups + g] : 0.f;
    float hat[H][V], d[H][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (here && pos[h] >= 0) {
        const P qx = *(const P*)((const T*)a.x.p + n * a.x.sb + pos[h] * a.x.st + ch[h]);
        const P qd = *(const P*)((const T*)a.dy.p + n * a.dy.sb + pos[h] * a.dy.st + ch[h]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float t = (qx.get(e) - mean) * rstd;
          const float dz = qd.get(e) * slope<SILU>(fmaf(t, w[h][e], b[h][e]));
          hat[h][e] = t;
          db[h][e] += dz;
          dw[h][e] = fmaf(dz, t, dw[h][e]);
          d[h][e] = dz * w[h][e];
          s1 += d[h][e];
          s2 = fmaf(d[h][e], t, s2);
        }
      }
    s1 = sum_of<WIDE>(s1, team, lds) * inv;
    s2 = sum_of<WIDE>(s2, team, lds) * inv;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (here && pos[h] >= 0) {
        P q;
#pragma unroll
        for (int e = 0; e < V; ++e) q.set(e, rstd * (d[h][e] - s1 - hat[h][e] * s2));
        *(P*)((T*)a.y + (n * a.p + pos[h]) * a.c + ch[h]) = q;
      }
  }
  if (a.dweight || a.dbias)
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (pos[h] >= 0) {
        float2* to = (float2*)a.chan + (id / a.groups * a.p + pos[h]) * a.c + ch[h];
#pragma unroll
        for (int e = 0; e < V; ++e) to[e] = make_float2(dw[h][e], db[h][e]);
      }
}

}  // namespace

hipError_t launch_norm_team_fwd(const NormArgs& a, hipStream_t s) {
  return for_kind(a.dtype, a.plan.v, a.act, [&](auto t, auto v, auto silu) {
    typedef decltype(t) T;
    constexpr int V = decltype(v)::value;
    constexpr bool SILU = decltype(silu)::value;
    const dim3 grid((unsigned)a.plan.blocks), block(kThreads);
    if (a.plan.held == 1 && a.plan.team <= 64)
      hipLaunchKernelGGL((norm_team_fwd_kernel<T, V, SILU, 1, false>), grid, block, 0, s, a);
    else if (a.plan.team <= 64)
      hipLaunchKernelGGL((norm_team_fwd_kernel<T, V, SILU, kTeamHeld, false>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((norm_team_fwd_kernel<T, V, SILU, kTeamHeld, true>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_team_bwd(const NormArgs& a, hipStream_t s) {
  return for_kind(a.dtype, a.plan.v, a.act, [&](auto t, auto v, auto silu) {
    typedef decltype(t) T;
    constexpr int V = decltype(v)::value;
    constexpr bool SILU = decltype(silu)::value;
    const dim3 grid((unsigned)a.plan.blocks), block(kThreads);
    if (a.plan.held == 1 && a.plan.team <= 64)
      hipLaunchKernelGGL((norm_team_bwd_kernel<T, V, SILU, 1, false>), grid, block, 0, s, a);
    else if (a.plan.team <= 64)
      hipLaunchKernelGGL((norm_team_bwd_kernel<T, V, SILU, kTeamHeldBwd, false>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((norm_team_bwd_kernel<T, V, SILU, kTeamHeldBwd, true>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace convnorm
