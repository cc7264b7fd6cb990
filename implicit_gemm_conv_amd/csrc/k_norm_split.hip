// k_norm_split.hip -- group norm over images and volumes: the sums of tiles of
// positions, and a second pass over x that writes the result.  The sums are joined at
// the second pass's beginning, or by a launch between.
//
// Bound by memory, x being read twice (a group of 56 x 56 x 8 channels is 50 KB of 16-byte
// pieces 512 bytes apart, so that no workgroup can hold whole lines of it): 32 images of
// 56 x 56 x 256, silu, bf16: sums 12.8 us (4.0 TB/s), result 29 (5.3 with what the caches
// hold); backward 29 and 37 (3.5 and 4.2 TB/s).
#include "norm_device.h"

namespace convnorm {

namespace {

constexpr int kLook = 4;  // rows a thread has in flight

// A workgroup's part of the problem: thread (col, row) owns the channels at `ch`
// and rows row, row + rw, ... of the tile.
struct Part {
  int n, tile, g0, slice, c0, width, rw, col, row, p0, p1;
  bool live;
};
template <int V>
__device__ __forceinline__ Part part_of(const NormArgs& a, unsigned b = blockIdx.x) {
  const Plan& pl = a.plan;
  Part t;
  const int cg = a.c / a.groups;
  const int cb = b % pl.cblocks;
  b /= pl.cblocks;
  t.tile = b % pl.tiles;
  t.n = b / pl.tiles;
  if (pl.slices == 1) {
    t.g0 = cb * pl.k;
    t.slice = 0;
    t.c0 = t.g0 * cg;
    t.width = min(pl.cw, a.c - t.c0);
  } else {
    t.g0 = cb / pl.slices;
    t.slice = cb % pl.slices;
    t.c0 = t.g0 * cg + t.slice * pl.cw;
    t.width = min(pl.cw, (t.g0 + 1) * cg - t.c0);
  }
  const int cv = pl.cw / V;
  t.rw = kThreads / cv;
  t.col = threadIdx.x % cv;
  t.row = threadIdx.x / cv;
  t.live = t.row < t.rw && t.col * V < t.width;
  t.p0 = t.tile * pl.per;
  t.p1 = min(t.p0 + pl.per, a.p);
  return t;
}

// Calls f(row pointer offset in rows, pack) for the thread's rows, kLook loads ahead.
template <typename T, int V, typename F>
__device__ __forceinline__ void walk(const Part& t, const Rows& r, int n, const F& f) {
  typedef Pack<T, V> P;
  const T* at = (const T*)r.p + n * r.sb + t.c0 + t.col * V;
  for (int p = t.p0 + t.row; p < t.p1; p += t.rw * kLook) {
    P q[kLook];
#pragma unroll
    for (int u = 0; u < kLook; ++u)
      if (p + u * t.rw < t.p1) q[u] = *(const P*)(at + (int64_t)(p + u * t.rw) * r.st);
#pragma unroll
    for (int u = 0; u < kLook; ++u)
      if (p + u * t.rw < t.p1) f(p + u * t.rw, q[u]);
  }
}

// Sums over the tile's channels of each of its groups, from a pair for each channel in LDS:
// put(group, lane of `of` lanes, first and last channel of the group in LDS).  Groups of few
// channels get a thread each, others a wave.
template <typename F>
__device__ __forceinline__ void each_group(const NormArgs& a, const Part& t, const F& f) {
  const int cg = a.plan.slices == 1 ? a.c / a.groups : t.width, groups = t.width / cg;
  if (cg <= 16) {
    for (int g = threadIdx.x; g < groups; g += kThreads) f(g, 0, 1, cg);
  } else {
    for (int g = threadIdx.x / 64; g < groups; g += kThreads / 64) f(g, threadIdx.x % 64, 64, cg);
  }
}

// What the rows of a workgroup hold for each of its channels: f(channel, the first row's pair, the distance of the
// rows' pairs), by one thread a channel.
template <int V, typename F>
__device__ __forceinline__ void add_rows(const NormArgs& a, const Part& t, const float (&x)[V], const float (&y)[V], float2* lds,
                                         const F& f) {
  if (t.live)
#pragma unroll
    for (int e = 0; e < V; ++e) lds[t.row * a.plan.cw + t.col * V + e] = make_float2(x[e], y[e]);
  __syncthreads();
  for (int c = threadIdx.x; c < t.width; c += kThreads) f(c, lds + c, a.plan.cw);
  __syncthreads();
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void norm_stats_kernel(NormArgs a) {
  __shared__ float2 lds[kThreads * V];
  const Part t = part_of<V>(a);
  const int each = max(t.p1 - t.p0, 0) / t.rw, over = max(t.p1 - t.p0, 0) % t.rw;
  const auto rows_of = [&](int row) { return (float)(each + (row < over)); };
  float m[V], s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) m[e] = s[e] = 0.f;
  if (t.live && t.p0 + t.row < t.p1) {
    // about the thread's own first row: the squares are of differences within the data's spread
    const Pack<T, V> first =
        *(const Pack<T, V>*)((const T*)a.x.p + t.n * a.x.sb + (t.p0 + t.row) * a.x.st + t.c0 + t.col * V);
    walk<T, V>(t, a.x, t.n, [&](int, const Pack<T, V>& q) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = q.get(e) - first.get(e);
        m[e] += d;
        s[e] = fmaf(d, d, s[e]);
      }
    });
    const float inv = 1.f / rows_of(t.row);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = m[e] * inv;
      s[e] = fmaf(-d, m[e], s[e]);
      m[e] = first.get(e) + d;
    }
  }
  // each channel's mean, then the squares about it
  const float all = 1.f / (float)max(t.p1 - t.p0, 1);
  const int filled = min(t.rw, t.p1 - t.p0);  // of the workgroup's rows
  add_rows<V>(a, t, m, s, lds, [&](int c, const float2* at, int ld) {
    float mean = 0.f, sq = 0.f;
    for (int r = 0; r < filled; ++r) mean = fmaf(rows_of(r) * all, at[r * ld].x - at[0].x, mean);
    mean += at[0].x;
    for (int r = 0; r < filled; ++r) {
      const float2 o = at[r * ld];
      const float d = o.x - mean;
      sq += fmaf(d * d, rows_of(r), o.y);
    }
    lds[c] = make_float2(mean, sq);
  });
  const float rows = (float)max(t.p1 - t.p0, 0);
  each_group(a, t, [&](int g, int lane, int of, int cg) {
    float mean = 0.f, sq = 0.f;
    for (int c = lane; c < cg; c += of) mean += lds[g * cg + c].x;
    mean = team_sum(mean, of) / (float)cg;
    for (int c = lane; c < cg; c += of) {
      const float2 o = lds[g * cg + c];
      const float d = o.x - mean;
      sq += fmaf(d * d, rows, o.y);
    }
    sq = team_sum(sq, of);
    if (lane == 0)
      ((float2*)a.part)[(((int64_t)t.n * a.groups + t.g0 + g) * a.plan.slices + t.slice) * a.plan.tiles + t.tile] =
          make_float2(mean, sq);
  });
}

// Values of part (slice, tile) of a group.
__device__ __forceinline__ double count_of(const NormArgs& a, int i) {
  const Plan& pl = a.plan;
  const int cg = a.c / a.groups, tile = i % pl.tiles, slice = i / pl.tiles;
  const int rows = min(pl.per, a.p - tile * pl.per), width = pl.slices == 1 ? cg : min(pl.cw, cg - slice * pl.cw);
  return (double)rows * width;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < kThreads / 64; ++w) v += lds[w];
  return v;
}

// Sum over `of` neighbouring threads, a power of two up to a wave, or the whole workgroup.
__device__ __forceinline__ double sum_over(double v, int of, double* lds) {
  if (of > 64) return block_sum(v, lds);
  for (int o = 1; o < of; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// The mean and 1 / deviation of a group from its parts, over `of` threads: the parts' means, then the squares about
// the whole mean.
__device__ __forceinline__ float2 join_stats(const NormArgs& a, int64_t group, int lane, int of, double* lds) {
  const int parts = a.plan.slices * a.plan.tiles;
  const float2* part = (const float2*)a.part + group * parts;
  const double all = (double)a.p * (a.c / a.groups);
  double sum = 0;
#pragma unroll 4
  for (int i = lane; i < parts; i += of) sum += count_of(a, i) * part[i].x;
  const double mean = sum_over(sum, of, lds) / all;
  sum = 0;
#pragma unroll 4
  for (int i = lane; i < parts; i += of) {
    const double d = part[i].x - mean;
    sum += part[i].y + count_of(a, i) * d * d;
  }
  sum = sum_over(sum, of, lds) / all;
  return make_float2((float)mean, (float)(1.0 / sqrt(sum + a.eps)));
}
// ... and the two means of the backward pass
__device__ __forceinline__ float2 join_means(const NormArgs& a, int64_t group, int lane, int of, double* lds) {
  const int parts = a.plan.slices * a.plan.tiles;
  const float2* part = (const float2*)a.part + group * parts;
  const double all = (double)a.p * (a.c / a.groups);
  double s1 = 0, s2 = 0;
#pragma unroll 4
  for (int i = lane; i < parts; i += of) {
    s1 += part[i].x;
    s2 += part[i].y;
  }
  s1 = sum_over(s1, of, lds);
  s2 = sum_over(s2, of, lds);
  return make_float2((float)(s1 / all), (float)(s2 / all));
}
// A workgroup's own groups: out[g] = f(the group's number, lane of `of` threads)
template <typename F>
__device__ __forceinline__ void join_groups(const NormArgs& a, const Part& t, float2* out, const F& f) {
  const int groups = a.plan.slices == 1 ? t.width / (a.c / a.groups) : 1, of = join_lanes(groups);
  for (int g0 = 0; g0 < groups; g0 += kThreads / of) {
    const int g = min(g0 + (int)threadIdx.x / of, groups - 1);
    const float2 o = f((int64_t)t.n * a.groups + t.g0 + g, threadIdx.x % of, of);
    if (threadIdx.x % of == 0) out[g] = o;
  }
  __syncthreads();
}

// One workgroup for each (n, group).
__global__ __launch_bounds__(kThreads) void norm_join_kernel(NormArgs a) {
  __shared__ double lds[kThreads / 64];
  const float2 o = join_stats(a, blockIdx.x, threadIdx.x, kThreads, lds);
  if (threadIdx.x == 0) {
    a.mean[blockIdx.x] = o.x;
    a.rstd[blockIdx.x] = o.y;
  }
}

// What a thread's channels are normalised with: the mean and 1 / deviation of their groups by f(group).
template <int V>
struct Channels {
  float mean[V], rstd[V], w[V], b[V];
  template <typename F>
  __device__ __forceinline__ Channels(const NormArgs& a, const Part& t, const F& f) {
    const int cg = a.c / a.groups;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = t.c0 + t.col * V + e;
      const float2 o = f(c / cg - t.g0);
      mean[e] = o.x;
      rstd[e] = o.y;
      w[e] = param(a.weight, a.param_f32, a.dtype, c, 1.f);
      b[e] = param(a.bias, a.param_f32, a.dtype, c, 0.f);
    }
  }
};
__device__ __forceinline__ float2 stats_in(const NormArgs& a, const Part& t, const float* mean, const float* rstd, int g) {
  const int64_t at = (int64_t)t.n * a.groups + t.g0 + g;
  return make_float2(mean[at], rstd[at]);
}

template <typename T, int V, bool SILU, bool JOINT>
__global__ __launch_bounds__(kThreads) void norm_apply_kernel(NormArgs a) {
  __shared__ float2 stats[JOINT ? 1 : kThreads * V];
  __shared__ double lds[kThreads / 64];
  const Part t = part_of<V>(a);
  if (!JOINT)
    join_groups(a, t, stats, [&](int64_t group, int lane, int of) {
      const float2 o = join_stats(a, group, lane, of, lds);
      if (lane == 0 && t.tile == 0 && t.slice == 0) {
        a.mean[group] = o.x;
        a.rstd[group] = o.y;
      }
      return o;
    });
  if (!t.live) return;
  const Channels<V> k(a, t, [&](int g) { return JOINT ? stats_in(a, t, a.mean, a.rstd, g) : stats[g]; });
  T* y = (T*)a.y + (int64_t)t.n * a.p * a.c + t.c0 + t.col * V;
  walk<T, V>(t, a.x, t.n, [&](int p, const Pack<T, V>& q) {
    Pack<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) o.set(e, activate<SILU>(fmaf((q.get(e) - k.mean[e]) * k.rstd[e], k.w[e], k.b[e])));
    *(Pack<T, V>*)(y + (int64_t)p * a.c) = o;
  });
}

// f(position, pieces of x and dy) for the thread's rows.
template <typename T, int V, typename F>
__device__ __forceinline__ void walk2(const NormArgs& a, const Part& t, const F& f) {
  typedef Pack<T, V> P;
  const T* x = (const T*)a.x.p + t.n * a.x.sb + t.c0 + t.col * V;
  const T* d = (const T*)a.dy.p + t.n * a.dy.sb + t.c0 + t.col * V;
  constexpr int look = kLook / 2;
  for (int p = t.p0 + t.row; p < t.p1; p += t.rw * look) {
    P q[look], r[look];
#pragma unroll
    for (int u = 0; u < look; ++u)
      if (p + u * t.rw < t.p1) {
        q[u] = *(const P*)(x + (int64_t)(p + u * t.rw) * a.x.st);
        r[u] = *(const P*)(d + (int64_t)(p + u * t.rw) * a.dy.st);
      }
#pragma unroll
    for (int u = 0; u < look; ++u)
      if (p + u * t.rw < t.p1) f(p + u * t.rw, q[u], r[u]);
  }
}

// For each channel of the tile the sums of dz xhat and dz, and from them, with the
// weights, the two sums of each group.
template <typename T, int V, bool SILU>
__global__ __launch_bounds__(kThreads) void norm_sums_kernel(NormArgs a) {
  __shared__ float2 lds[kThreads * V];
  const Part t = part_of<V>(a);
  float dw[V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) dw[e] = db[e] = 0.f;
  if (t.live) {
    const Channels<V> k(a, t, [&](int g) { return stats_in(a, t, a.mean_in, a.rstd_in, g); });
    walk2<T, V>(a, t, [&](int, const Pack<T, V>& q, const Pack<T, V>& r) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hat = (q.get(e) - k.mean[e]) * k.rstd[e];
        const float dz = r.get(e) * slope<SILU>(fmaf(hat, k.w[e], k.b[e]));
        db[e] += dz;
        dw[e] = fmaf(dz, hat, dw[e]);
      }
    });
  }
  float2* to = (float2*)a.chan + ((int64_t)t.n * a.plan.tiles + t.tile) * a.c + t.c0;
  add_rows<V>(a, t, dw, db, lds, [&](int c, const float2* at, int ld) {
    float2 o = at[0];
    for (int r = 1; r < t.rw; ++r) {
      o.x += at[r * ld].x;
      o.y += at[r * ld].y;
    }
    const float w = param(a.weight, a.param_f32, a.dtype, t.c0 + c, 1.f);
    to[c] = o;
    lds[c] = make_float2(o.x * w, o.y * w);
  });
  each_group(a, t, [&](int g, int lane, int of, int cg) {
    float s1 = 0.f, s2 = 0.f;
    for (int c = lane; c < cg; c += of) {
      s2 += lds[g * cg + c].x;
      s1 += lds[g * cg + c].y;
    }
    s1 = team_sum(s1, of);
    s2 = team_sum(s2, of);
    if (lane == 0)
      ((float2*)a.part)[(((int64_t)t.n * a.groups + t.g0 + g) * a.plan.slices + t.slice) * a.plan.tiles + t.tile] =
          make_float2(s1, s2);
  });
}

// dweight and dbias of kCols channels a workgroup, from the sums of all tiles.
constexpr int kCols = 8;
__device__ void columns(const NormArgs& a, int block, double* lds) {
  const int c = block * kCols + threadIdx.x % kCols, lane = threadIdx.x / kCols;
  double dw = 0, db = 0;
  if (c < a.c)
#pragma unroll 8
    for (int64_t r = lane; r < a.plan.rows; r += kThreads / kCols) {
      const float2 o = ((const float2*)a.chan)[r * a.c + c];
      dw += o.x;
      db += o.y;
    }
  double* mine = lds + threadIdx.x * 2;
  mine[0] = dw;
  mine[1] = db;
  for (int half = kThreads / kCols / 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (lane < half) {
      mine[0] += mine[half * kCols * 2];
      mine[1] += mine[half * kCols * 2 + 1];
    }
  }
  if (lane == 0 && c < a.c) {
    if (a.dweight) a.dweight[c] = (float)mine[0];
    if (a.dbias) a.dbias[c] = (float)mine[1];
  }
}

__global__ __launch_bounds__(kThreads) void norm_columns_kernel(NormArgs a) {
  __shared__ double lds[2 * kThreads];
  columns(a, blockIdx.x, lds);
}

// The first N * groups workgroups: the two means of an (n, group); the others: the parameters' columns.
__global__ __launch_bounds__(kThreads) void norm_join_bwd_kernel(NormArgs a) {
  __shared__ double lds[2 * kThreads];
  const int64_t slabs = (int64_t)a.n * a.groups;
  if (blockIdx.x >= slabs) return columns(a, (int)(blockIdx.x - slabs), lds);
  const float2 o = join_means(a, blockIdx.x, threadIdx.x, kThreads, lds);
  if (threadIdx.x == 0) ((float2*)a.two)[blockIdx.x] = o;
}

// Not JOINT: the first `cols` workgroups add the parameters' columns, the others write dx.
template <typename T, int V, bool SILU, bool JOINT>
__global__ __launch_bounds__(kThreads) void norm_apply_bwd_kernel(NormArgs a, int cols) {
  __shared__ union {
    float2 means[JOINT ? 1 : kThreads * V];
    double sums[JOINT ? 1 : 2 * kThreads];
  } s;
  __shared__ double lds[kThreads / 64];
  if (!JOINT && (int)blockIdx.x < cols) return columns(a, blockIdx.x, s.sums);
  const Part t = part_of<V>(a, blockIdx.x - (JOINT ? 0 : cols));
  if (!JOINT) join_groups(a, t, s.means, [&](int64_t group, int lane, int of) { return join_means(a, group, lane, of, lds); });
  if (!t.live) return;
  const int cg = a.c / a.groups;
  const Channels<V> k(a, t, [&](int g) { return stats_in(a, t, a.mean_in, a.rstd_in, g); });
  float s1[V], s2[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int g = (t.c0 + t.col * V + e) / cg - t.g0;
    const float2 o = JOINT ? ((const float2*)a.two)[(int64_t)t.n * a.groups + t.g0 + g] : s.means[g];
    s1[e] = o.x;
    s2[e] = o.y;
  }
  T* dx = (T*)a.y + (int64_t)t.n * a.p * a.c + t.c0 + t.col * V;
  walk2<T, V>(a, t, [&](int p, const Pack<T, V>& q, const Pack<T, V>& r) {
    Pack<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float hat = (q.get(e) - k.mean[e]) * k.rstd[e];
      const float d = r.get(e) * slope<SILU>(fmaf(hat, k.w[e], k.b[e])) * k.w[e];
      o.set(e, k.rstd[e] * (d - s1[e] - hat * s2[e]));
    }
    *(Pack<T, V>*)(dx + (int64_t)p * a.c) = o;
  });
}

}  // namespace

hipError_t launch_norm_columns(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_columns_kernel, dim3((a.c + kCols - 1) / kCols), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  return for_kind(a.dtype, a.plan.v, a.act, [&](auto t, auto v, auto silu) {
    typedef decltype(t) T;
    constexpr int V = decltype(v)::value;
    constexpr bool SILU = decltype(silu)::value;
    const dim3 grid((unsigned)a.plan.blocks), block(kThreads);
    hipLaunchKernelGGL((norm_stats_kernel<T, V>), grid, block, 0, s, a);
    const dim3 slabs((unsigned)((int64_t)a.n * a.groups));
    if (a.plan.joint) hipLaunchKernelGGL(norm_join_kernel, slabs, block, 0, s, a);
    hipLaunchKernelGGL((a.plan.joint ? norm_apply_kernel<T, V, SILU, true> : norm_apply_kernel<T, V, SILU, false>), grid, block, 0,
                       s, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  return for_kind(a.dtype, a.plan.v, a.act, [&](auto t, auto v, auto silu) {
    typedef decltype(t) T;
    constexpr int V = decltype(v)::value;
    constexpr bool SILU = decltype(silu)::value;
    const dim3 block(kThreads);
    const int cols = a.dweight || a.dbias ? (a.c + kCols - 1) / kCols : 0;
    hipLaunchKernelGGL((norm_sums_kernel<T, V, SILU>), dim3((unsigned)a.plan.blocks), block, 0, s, a);
    if (a.plan.joint) {
      hipLaunchKernelGGL(norm_join_bwd_kernel, dim3((unsigned)((int64_t)a.n * a.groups + cols)), block, 0, s, a);
      hipLaunchKernelGGL((norm_apply_bwd_kernel<T, V, SILU, true>), dim3((unsigned)a.plan.blocks), block, 0, s, a, 0);
    } else {
      hipLaunchKernelGGL((norm_apply_bwd_kernel<T, V, SILU, false>), dim3((unsigned)(a.plan.blocks + cols)), block, 0, s, a, cols);
    }
    return hipGetLastError();
  });
}

}  // namespace convnorm
