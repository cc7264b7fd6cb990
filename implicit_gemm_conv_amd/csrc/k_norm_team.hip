// k_norm_team.hip -- group norm where an (n, group) fits the registers of a
// team of lanes: rows normalised head by head, small images.  x is read once,
// the mean and the variance about it are taken from what is held.
//
// 16384 rows of 16 groups of 128 channels, silu, bf16: forward 43-46 us (2.9 TB/s), backward 53-55
// and 7 for the parameters' columns (3.8 TB/s).  Bound by vector work (busy 66% and 60%: conversions,
// the activation, sums over lanes) beside memory.
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
// position i / (pieces a position), channels of piece i % (pieces a position).  A team
// keeps its group of channels, whose parameters stay in registers, and walks over n; the
// next n's pieces are loaded before this one's are worked on.
template <typename T, int V, int H>
struct Walk {
  const NormArgs& a;
  int lane, g, pos[H], ch[H];  // pos: -1 where the lane has no such piece
  int64_t first, step, turns;  // n's; every team of a workgroup makes as many turns (wide teams wait for each other)
  float w[H][V], b[H][V];

  __device__ __forceinline__ Walk(const NormArgs& a_) : a(a_) {
    const int team = a.plan.team, cg = a.c / a.groups, wide = cg / V, pieces = wide * a.p;
    const int64_t id = (int64_t)blockIdx.x * (kThreads / team) + threadIdx.x / team;
    step = a.plan.step;
    turns = (a.n + step - 1) / step;
    lane = threadIdx.x % team;
    g = (int)(id % a.groups);
    first = id / a.groups;
    const bool live = first < step;
    if (!live) first = a.n;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int i = lane + h * team;
      pos[h] = live && i < pieces ? i / wide : -1;
      ch[h] = g * cg + (i < pieces ? i % wide * V : 0);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[h][e] = param(a.weight, a.param_f32, a.dtype, ch[h] + e, 1.f);
        b[h][e] = param(a.bias, a.param_f32, a.dtype, ch[h] + e, 0.f);
      }
    }
  }
  __device__ __forceinline__ int64_t n(int64_t turn) const { return first + turn * step; }
  __device__ __forceinline__ bool has(int h, int64_t turn) const { return pos[h] >= 0 && n(turn) < a.n; }
  __device__ __forceinline__ void load(const Rows& x, int64_t turn, Pack<T, V> (&q)[H]) const {
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (has(h, turn)) q[h] = *(const Pack<T, V>*)((const T*)x.p + n(turn) * x.sb + pos[h] * x.st + ch[h]);
  }
  __device__ __forceinline__ void store(int h, int64_t turn, const Pack<T, V>& q) const {
    *(Pack<T, V>*)((T*)a.y + (n(turn) * a.p + pos[h]) * a.c + ch[h]) = q;
  }
};

template <typename T, int V, bool SILU, int H, bool WIDE>
__global__ __launch_bounds__(kThreads) void norm_team_fwd_kernel(NormArgs a) {
  __shared__ float lds[kThreads / 64];
  const int team = a.plan.team, cg = a.c / a.groups;
  const float inv = 1.f / (float)max(cg * a.p, 1);
  typedef Pack<T, V> P;
  const Walk<T, V, H> t(a);
  P q[H], ahead[H];
  t.load(a.x, 0, ahead);
  for (int64_t turn = 0; turn < t.turns; ++turn) {
#pragma unroll
    for (int h = 0; h < H; ++h) q[h] = ahead[h];
    t.load(a.x, turn + 1, ahead);
    float v[H][V], sum = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (t.has(h, turn))
#pragma unroll
        for (int e = 0; e < V; ++e) sum += v[h][e] = q[h].get(e);
    // about a first mean, whose own rounding the sum of the differences then takes out
    float mean = sum_of<WIDE>(sum, team, lds) * inv, off = 0.f;
    sum = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (t.has(h, turn))
#pragma unroll
        for (int e = 0; e < V; ++e) {
          v[h][e] -= mean;
          off += v[h][e];
          sum = fmaf(v[h][e], v[h][e], sum);
        }
    off = sum_of<WIDE>(off, team, lds) * inv;
    mean += off;
    const float var = fmaf(-off, off, sum_of<WIDE>(sum, team, lds) * inv);
    const float rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + a.eps);  // NaN stays
    if (t.lane == 0 && t.n(turn) < a.n) {
      a.mean[t.n(turn) * a.groups + t.g] = mean;
      a.rstd[t.n(turn) * a.groups + t.g] = rstd;
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (t.has(h, turn)) {
        P o;
#pragma unroll
        for (int e = 0; e < V; ++e) o.set(e, activate<SILU>(fmaf((v[h][e] - off) * rstd, t.w[h][e], t.b[h][e])));
        t.store(h, turn, o);
      }
  }
}

// The same cut.  A lane's sums for the parameters stay in registers too; they are left, a
// row for each position of each team, to the columns' kernel.
template <typename T, int V, bool SILU, int H, bool WIDE>
__global__ __launch_bounds__(kThreads) void norm_team_bwd_kernel(NormArgs a) {
  __shared__ float lds[kThreads / 64];
  const int team = a.plan.team, cg = a.c / a.groups;
  const float inv = 1.f / (float)max(cg * a.p, 1);
  typedef Pack<T, V> P;
  const Walk<T, V, H> t(a);
  float dw[H][V], db[H][V];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[h][e] = db[h][e] = 0.f;
  P x[H], dy[H], x_next[H], dy_next[H];
  float mean_next = 0.f, rstd_next = 0.f;
  const auto load = [&](int64_t turn) {
    t.load(a.x, turn, x_next);
    t.load(a.dy, turn, dy_next);
    if (t.n(turn) < a.n) {
      mean_next = a.mean_in[t.n(turn) * a.groups + t.g];
      rstd_next = a.rstd_in[t.n(turn) * a.groups + t.g];
    }
  };
  load(0);
  for (int64_t turn = 0; turn < t.turns; ++turn) {
    const float mean = mean_next, rstd = rstd_next;
#pragma unroll
    for (int h = 0; h < H; ++h) x[h] = x_next[h], dy[h] = dy_next[h];
    load(turn + 1);
    float hat[H][V], d[H][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (t.has(h, turn))
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float at = (x[h].get(e) - mean) * rstd;
          const float dz = dy[h].get(e) * slope<SILU>(fmaf(at, t.w[h][e], t.b[h][e]));
          hat[h][e] = at;
          db[h][e] += dz;
          dw[h][e] = fmaf(dz, at, dw[h][e]);
          d[h][e] = dz * t.w[h][e];
          s1 += d[h][e];
          s2 = fmaf(d[h][e], at, s2);
        }
    s1 = sum_of<WIDE>(s1, team, lds) * inv;
    s2 = sum_of<WIDE>(s2, team, lds) * inv;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (t.has(h, turn)) {
        P o;
#pragma unroll
        for (int e = 0; e < V; ++e) o.set(e, rstd * (d[h][e] - s1 - hat[h][e] * s2));
        t.store(h, turn, o);
      }
  }
  if (a.dweight || a.dbias)
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (t.pos[h] >= 0) {
        float2* to = (float2*)a.chan + (t.first * a.p + t.pos[h]) * a.c + t.ch[h];
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
    else if (a.plan.held == 1)
      hipLaunchKernelGGL((norm_team_fwd_kernel<T, V, SILU, 1, true>), grid, block, 0, s, a);
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
    else if (a.plan.held == 1)
      hipLaunchKernelGGL((norm_team_bwd_kernel<T, V, SILU, 1, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((norm_team_bwd_kernel<T, V, SILU, kTeamHeldBwd, true>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace convnorm
