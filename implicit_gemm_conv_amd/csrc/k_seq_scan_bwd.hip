// k_seq_scan_bwd.hip -- gated linear recurrence, backward, in one pass.
//
// With r = sigmoid(gate_r), i = sigmoid(gate_i), u = decay * softplus(lam) * r,
// a = e^-u, m = sqrt(1 - a^2), h_t = a h_{t-1} + m i x_t, and g_t the whole
// gradient of h_t:
//
//   c_t = a_t g_t,  g_t = dy_t + c_{t+1}     (c_t = 0 where t begins a sequence)
//   dx = g m i,   dgate_i = g m i x (1 - i)
//   e = g u a (a i x / m - h_{t-1}),  dgate_r = e (1 - r)
//   dlam = (sigmoid(lam) / softplus(lam)) sum e,   dh0 = c_0
//
// (dm/du = a^2 / m, and u / m goes to zero with u.)  Both recurrences, h forward
// from the state kept before each 64 rows and c backward from the sequence's
// end, go through the same tile: a workgroup of 8 waves takes 64 rows by 64 V
// channels, a wave 8 rows, a lane V channels of those.  The lane composes its
// rows into one step of h and one of c; the waves' steps are composed through
// LDS, and the tiles' steps of c through memory from the last tile to the first
// (seq_carry.h).  Then the lane runs c up its rows, with r, i, m i and
// a i x / m - h_{t-1} of each value held in registers, and stores the three
// gradients; a is computed again from r, which is cheaper than the registers it
// would take (at 128, two workgroups fit a compute unit).  Each input is read once, each gradient written once: memory
// bound, 4 elements (or 1 element and 3 bytes) in and 3 out a value.
//
// 4x4096x2048 bf16 from 8 bits takes 123 to 127 us, the vector ALU busy 62% of it; a
// workgroup lives 13.9 us, 8.5 of them waiting (ticket 0.7, loads 3.0, its waves 1.4 and
// 1.7, look-back 1.7).  3x1999x321 fp32, one channel a lane, takes 19 us.  V is 2
// where C, strides and alignment allow pairs of 16-bit values: with 1 the former
// takes 139 us, and 64x100x512 fp16 18.7 instead of 18.0.
#include "seq_carry.h"

namespace convseq {

namespace {

constexpr int kWaves = 8;
constexpr int kRows = 8;  // of a wave
constexpr int kTile = kWaves * kRows;
static_assert(kTile == kEvery, "a tile starts from a kept state");

template <typename T, int V, bool STARTS, bool KEPT>
__global__ __launch_bounds__(kWaves * 64, V == 1 ? 6 : 4) void seq_scan_bwd_kernel(ScanArgs a, int cols, int tiles) {
  __shared__ Carry down[kWaves][64 * V], up[kWaves][64 * V];
  __shared__ float entry[64 * V], rates[64 * V];
  __shared__ Gathered<V, kWaves> gathered;
  __shared__ float sums[kWaves][64 * V];
  __shared__ int ticket;
  typedef Pack<T, V> P;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int columns = cols * a.b, column = (blockIdx.x + blockIdx.x / columns) % columns;
  const int turn = tiles > 1 ? take_ticket(a.work, column, &ticket) : 0;
  const int tile = tiles - 1 - turn;  // from the end of the sequence
  const int b = column / cols;
  const int ch = (column % cols * 64 + lane) * V;
  const int chl = min(ch, a.c - V);  // lanes past the last channel read it again
  const bool own = ch < a.c;
  const int t0 = tile * kTile + wave * kRows;
  const int n = min(max(a.t - t0, 0), kRows);  // rows of this wave

  P ry[kRows], raw[3][kRows];
  Half<V> q[3];
  float scale[3][V];
  // rows past the last read it again
  const int64_t row = min(t0, a.t - 1);
  const auto walk = [&](const Rows& r) {
    return RowWalk((const T*)r.p + b * r.sb + row * r.st, r.st * (int64_t)sizeof(T));
  };
  {
    uint32_t offset = (uint32_t)chl * sizeof(T);
    renew(offset);
    RowWalk wy = walk(a.dy), wx = walk(a.x), wr = walk(a.r), wi = walk(a.i);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      ry[j] = wy.load<P>(offset);
      wy.step(j + 1 < n);
      if (KEPT) continue;
      raw[0][j] = wx.load<P>(offset);
      raw[1][j] = wr.load<P>(offset);
      raw[2][j] = wi.load<P>(offset);
      wx.step(j + 1 < n);
      wr.step(j + 1 < n);
      wi.step(j + 1 < n);
    }
  }
  if (KEPT) {
    const int groups = (a.t + kGroup - 1) / kGroup;
    const int64_t at = (int64_t)b * groups + min(t0 / kGroup, groups - 1);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      q[k] = half_group<V>(a.kept[k], at, t0 / kRows % 2, a.c, chl);
      group_scales<V>(a.kept[k], at, a.c, chl, scale[k]);
#pragma unroll
      for (int i = 0; i < V; ++i) scale[k][i] *= k > 0 ? -kLog2e : 1.f;
    }
  }
  // x, and the gates' logits times -log2 e
  const auto value = [&](int k, int j, int i) -> float {
    if (KEPT) return q[k].get(i, j) * scale[k][i];
    return k > 0 ? -kLog2e * raw[k][j].get(i) : raw[k][j].get(i);
  };
  uint32_t first = 0;  // bit j: row t0 + j begins a sequence
  if (STARTS) first = (uint32_t)__ballot(lane < n && a.starts[(int64_t)b * a.t + t0 + lane]);
  const int pieces = (a.t + kEvery - 1) / kEvery;
  float h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = load_at<float>(a.states_in + ((int64_t)b * pieces + tile) * a.c, (uint32_t)(chl + i) * 4);
  if (wave < V) {
    const int k = wave * 64 + lane;
    rates[k] = a.decay * softplus(a.lam[min(column % cols * 64 * V + k, a.c - 1)]);
  }
  lds_barrier();
  Rate rate[V];
#pragma unroll
  for (int i = 0; i < V; ++i) rate[i] = rate_of(rates[lane * V + i]);

  // gates, and this wave's steps of h and c
  float rv[kRows][V], iv[kRows][V], mi[kRows][V], kv[kRows][V];  // r, i, m i, a i x / m less what is known of h_{t-1}
  Carry step[V];
#pragma unroll
  for (int i = 0; i < V; ++i) step[i] = Carry{1.f, 0.f};
  float sent[V];  // what the rows' dy make of c before the first row
#pragma unroll
  for (int i = 0; i < V; ++i) sent[i] = 0.f;
#pragma unroll
  for (int j = 0; j < kRows; ++j)
    if (j < n) {
      const bool begins = STARTS && (first >> j & 1);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float x = value(0, j, i);
        const Gate g = gates(value(1, j, i), value(2, j, i), rate[i]);
        const float rs = inv_sqrt(g.t), m = g.t * rs, v = g.i * x, in = m * v;
        rv[j][i] = g.r;
        iv[j][i] = g.i;
        mi[j][i] = m * g.i;
        kv[j][i] = g.a * rs * v;
        if (!begins) kv[j][i] -= step[i].h;
        const float h = fmaf(g.a, step[i].h, in);
        step[i] = Carry{begins ? -0.f : positive(step[i].a * g.a), begins ? in : h};
        // rows from a start on send nothing up (asked of the starts, not of the
        // product, which a NaN behind the start may have taken)
        if (!STARTS || (first & ((2u << j) - 1u)) == 0) sent[i] = fmaf(step[i].a, ry[j].get(i), sent[i]);
      }
    }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    down[wave][lane * V + i] = step[i];
    up[wave][lane * V + i] = Carry{STARTS && first ? -0.f : step[i].a, sent[i]};
  }
  lds_barrier();

  // wave 0 has the tile's step of c, and gets the c after the tile
  float c[V];
  Carry whole[V];
  const CarrySpace space = carry_space(a.work, tiles - 1, cols * a.b);
  uint64_t* words = space.words + (int64_t)column * 64 * V;
  uint32_t* flags = space.flags + (int64_t)column * (tiles - 1);
  const int64_t stride = (int64_t)cols * a.b * 64 * V;
  uint64_t* mine = words + turn * stride;  // and the lane's from lane * V
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) whole[i] = Carry{1.f, 0.f};
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w)
#pragma unroll
      for (int i = 0; i < V; ++i) whole[i] = compose(whole[i], up[w][lane * V + i]);
    if (turn > 0 && tile > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) publish(mine + (uint32_t)(lane * V + i), whole[i]);
      if (lane == 0) raise_flag(flags + turn, 1);
    }
  }
  // The state before these rows reaches row j as the product of the a before it,
  // e^-(sum of u), up to the first start: kv becomes a i x / m - h_{j-1}, while the
  // tiles before this one finish.
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = apply(down[w][lane * V + i], h[i]);
  const int reached = STARTS && first ? min(n, __builtin_ctz(first)) : n;
  float open[V];
#pragma unroll
  for (int i = 0; i < V; ++i) open[i] = 0.f;
#pragma unroll
  for (int j = 0; j < kRows; ++j)
    if (j < reached) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        kv[j][i] = fmaf(-__builtin_amdgcn_exp2f(rate[i].log2 * open[i]), h[i], kv[j][i]);
        open[i] += rv[j][i];
      }
    }

  if (turn == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = a.dh_last ? a.dh_last[(int64_t)b * a.c + chl + i] : 0.f;
  } else {
    look_back<V, kWaves>(words, stride, flags, turn, wave, lane, wave == 0, gathered, c);
  }
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float after = apply(whole[i], c[i]);
      if (tile > 0)
        publish(mine + (uint32_t)(lane * V + i), Carry{__uint_as_float(kWhole), after});
      else if (a.dh0 && own)
        a.dh0[(int64_t)b * a.c + ch + i] = after;
      entry[lane * V + i] = c[i];
    }
    if (tile > 0 && lane == 0) raise_flag(flags + turn, 2);
  }

  lds_barrier();

  // c up the rows
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = entry[lane * V + i];
    sum[i] = 0.f;
  }
  for (int w = kWaves - 1; w > wave; --w)
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = apply(up[w][lane * V + i], c[i]);
  const int64_t out = ((int64_t)b * a.t + t0) * a.c;
  if (KEPT) renew(q[0]);
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    renew(ry[j]);
    if (!KEPT) renew(raw[0][j]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    renew(rate[i].u);
    renew(rate[i].log2);
  }
  const auto run_up = [&](auto whole) {
    uint32_t offset = (uint32_t)ch * sizeof(T);
    renew(offset);
    const int64_t end = out + (int64_t)(kRows - 1) * a.c, up = -(int64_t)a.c * (int64_t)sizeof(T);
    RowWalk px((T*)a.dx + end, up), pr((T*)a.dr + end, up), pi((T*)a.di + end, up);
#pragma unroll
    for (int j = kRows - 1; j >= 0; --j) {
      if (decltype(whole)::value || j < n) {
        P dx, dr, di;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float g = ry[j].get(i) + c[i];
          const float gm = g * mi[j][i], ga = g * positive(__builtin_amdgcn_exp2f(rate[i].log2 * rv[j][i]));
          // x (1 - i), x's power of two in the subtraction's place
          const float xi = KEPT ? q[0].get(i, j) * fmaf(-scale[0][i], iv[j][i], scale[0][i])
                                : raw[0][j].get(i) * (1.f - iv[j][i]);
          const float e = ga * (rate[i].u * rv[j][i]) * kv[j][i];
          dx.set(i, gm);
          di.set(i, gm * xi);
          dr.set(i, e * (1.f - rv[j][i]));
          sum[i] += e;
          c[i] = STARTS && (first >> j & 1) ? 0.f : ga;
        }
        px.store(offset, dx);
        pr.store(offset, dr);
        pi.store(offset, di);
      }
      px.step();
      pr.step();
      pi.step();
      if (decltype(whole)::value) __builtin_amdgcn_sched_barrier(0);  // rows worked on together cost registers
    }
  };
  if (own) {
    if (n == kRows)
      run_up(Yes{});
    else
      run_up(No{});
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[wave][lane * V + i] = sum[i];
  lds_barrier();
  if (wave == 0 && own) {
    float* part = a.parts + ((int64_t)tile * a.b + b) * a.c + ch;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += sums[w][lane * V + i];
      part[i] = s;
    }
  }
}

// dlam from the tiles' sums: 32 channels a workgroup, 32 threads a channel that
// each add every 32nd part, then the threads' sums in order.
__global__ __launch_bounds__(1024) void seq_scan_sum_kernel(const float* parts, int64_t count, int c, const float* lam,
                                                            float* dlam) {
  __shared__ float s[32][33];
  const int ch = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float v = 0.f;
  if (ch < c)
    for (int64_t p = k; p < count; p += 32) v += parts[p * c + ch];
  s[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k == 0 && ch < c) {
    v = 0.f;
    for (int j = 0; j < 32; ++j) v += s[j][threadIdx.x];
    dlam[ch] = v * channel_unit(lam[ch]);
  }
}

// No rows: the state's gradient passes through.
__global__ __launch_bounds__(256) void scan_pass_kernel(const float* dh_last, int64_t n, float* dh0) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) dh0[i] = dh_last ? dh_last[i] : 0.f;
}

int tiles_of(int t) { return (t + kTile - 1) / kTile; }

template <typename T, int V, bool STARTS, bool KEPT>
hipError_t run(ScanArgs a, hipStream_t s) {
  const int cols = (a.c + 64 * V - 1) / (64 * V), tiles = tiles_of(a.t);
  const int64_t carry = tiles > 1 ? carry_bytes(tiles - 1, (int64_t)cols * a.b, 64 * V) : 0;
  if (tiles > 1) {
    const hipError_t e = carry_clear(a.work, carry, s);
    if (e != hipSuccess) return e;
  }
  a.parts = (float*)((char*)a.work + carry);
  hipLaunchKernelGGL((seq_scan_bwd_kernel<T, V, STARTS, KEPT>), dim3((unsigned)(cols * a.b * tiles)),
                     dim3(kWaves * 64), 0, s, a, cols, tiles);
  hipLaunchKernelGGL(seq_scan_sum_kernel, dim3((a.c + 31) / 32), dim3(1024), 0, s,
                     (const float*)a.parts, (int64_t)tiles * a.b, a.c, a.lam, a.dlam);
  return hipGetLastError();
}
template <typename T, int V>
hipError_t run_as(const ScanArgs& a, hipStream_t s) {
  if (a.starts) return a.kept[0].q ? run<T, V, true, true>(a, s) : run<T, V, true, false>(a, s);
  return a.kept[0].q ? run<T, V, false, true>(a, s) : run<T, V, false, false>(a, s);
}
template <typename T>
hipError_t run_16(const ScanArgs& a, hipStream_t s) {
  bool wide = a.c % 2 == 0 && pieces(a.dy, 4, 2) && ((uintptr_t)a.dx | (uintptr_t)a.dr | (uintptr_t)a.di) % 4 == 0 &&
              ((uintptr_t)a.kept[0].e | (uintptr_t)a.kept[1].e | (uintptr_t)a.kept[2].e) % 2 == 0;
  if (!a.kept[0].q) wide = wide && pieces(a.x, 4, 2) && pieces(a.r, 4, 2) && pieces(a.i, 4, 2);
  return wide ? run_as<T, 2>(a, s) : run_as<T, 1>(a, s);
}

}  // namespace

// The carry for whichever of the two column widths needs more, and the tiles' sums.
int64_t scan_bwd_work_bytes(int b, int t, int c) {
  const int64_t tiles = tiles_of(t);
  if (tiles == 0 || b == 0) return 0;
  const int64_t narrow = carry_bytes(tiles - 1, (int64_t)b * ((c + 63) / 64), 64);
  const int64_t wide = carry_bytes(tiles - 1, (int64_t)b * ((c + 127) / 128), 128);
  return (narrow > wide ? narrow : wide) + tiles * b * c * 4;
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s) {
  if (a.t == 0 || a.b == 0) {
    const int64_t n = (int64_t)a.b * a.c;
    if (a.dh0 && n > 0)
      hipLaunchKernelGGL(scan_pass_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.dh_last, n, a.dh0);
    hipLaunchKernelGGL(seq_scan_sum_kernel, dim3((a.c + 31) / 32), dim3(1024), 0, s, (const float*)nullptr, (int64_t)0,
                       a.c, a.lam, a.dlam);
    return hipGetLastError();
  }
  if (a.dtype == convfwd::kF32) return run_as<float, 1>(a, s);
  if (a.dtype == convfwd::kF16) return run_16<_Float16>(a, s);
  return run_16<__bf16>(a, s);
}

}  // namespace convseq
