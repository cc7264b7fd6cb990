// k_seq_scan_fwd.hip -- gated linear recurrence, forward, in one pass over the
// inputs.
//
//   r = sigmoid(gate_r), i = sigmoid(gate_i), u = decay * softplus(lam) * r, a = e^-u
//   h_t = a_t h_{t-1} + sqrt(1 - a^2) i x_t
//
// A workgroup of 8 waves takes a tile of 128 rows by 64 V channels, a wave 16
// rows of it, a lane V channels of those rows.  The lane composes its rows into
// one step h -> A h + H, the waves' steps are composed through LDS, the tiles'
// through memory (seq_carry.h), and with the state before its rows known the
// lane runs the recurrence over the a and m v it still holds.  Each input is
// read once and y written once: memory bound, 4 elements a value.
#include "seq_carry.h"

namespace convseq {

namespace {

constexpr int kWaves = 8;
constexpr int kTile = kWaves * kGroup;  // rows

template <typename T, int V, bool STARTS, bool KEEP>
__global__ __launch_bounds__(kWaves * 64, V == 1 ? 6 : 4) void seq_scan_fwd_kernel(ScanArgs a, int cols, int tiles) {
  __shared__ Carry totals[kWaves][64 * V];
  __shared__ float entry[64 * V], rates[64 * V];
  __shared__ Gathered<V, kWaves> gathered;
  __shared__ int ticket;
  typedef Pack<T, V> P;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int columns = cols * a.b, column = (blockIdx.x + blockIdx.x / columns) % columns;
  const int tile = tiles > 1 ? take_ticket(a.work, column, &ticket) : 0;
  const int b = column / cols;
  const int ch = (column % cols * 64 + lane) * V;
  const int chl = min(ch, a.c - V);  // lanes past the last channel read it again
  const bool own = ch < a.c;
  const int t0 = tile * kTile + wave * kGroup;
  const int n = min(max(a.t - t0, 0), kGroup);  // rows of this wave

  const uint32_t offset = (uint32_t)chl * sizeof(T);
  const T* px = (const T*)a.x.p + b * a.x.sb;
  const T* pr = (const T*)a.r.p + b * a.r.sb;
  const T* pi = (const T*)a.i.p + b * a.i.sb;
  P rx[kGroup], rr[kGroup], ri[kGroup];
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    const int64_t t = min(t0 + j, a.t - 1);  // rows past the last read it again
    rx[j] = load_at<P>(px + t * a.x.st, offset);
    rr[j] = load_at<P>(pr + t * a.r.st, offset);
    ri[j] = load_at<P>(pi + t * a.i.st, offset);
  }
  uint32_t first = 0;  // bit j: row t0 + j begins a sequence
  if (STARTS) first = (uint32_t)__ballot(lane < n && a.starts[(int64_t)b * a.t + t0 + lane]);
  if (wave < V) {
    const int k = wave * 64 + lane;
    rates[k] = a.decay * softplus(a.lam[min(column % cols * 64 * V + k, a.c - 1)]);
  }
  lds_barrier();
  Rate rate[V];
#pragma unroll
  for (int i = 0; i < V; ++i) rate[i] = rate_of(rates[lane * V + i]);

  if (KEEP && n > 0 && own) {
    const int64_t at = (int64_t)b * ((a.t + kGroup - 1) / kGroup) + t0 / kGroup;
    keep_group<T, V>(rx, n, a.kept[0], at, a.c, ch);
    keep_group<T, V>(rr, n, a.kept[1], at, a.c, ch);
    keep_group<T, V>(ri, n, a.kept[2], at, a.c, ch);
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      renew(rx[j]);
      renew(rr[j]);
      renew(ri[j]);
    }
  }

  float av[kGroup][V], in[kGroup][V];
  Carry total[V];
#pragma unroll
  for (int i = 0; i < V; ++i) total[i] = Carry{1.f, 0.f};
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < n) {
      const bool begins = STARTS && (first >> j & 1);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Gate g = gates(-kLog2e * rr[j].get(i), -kLog2e * ri[j].get(i), rate[i]);
        av[j][i] = g.a;
        in[j][i] = __builtin_amdgcn_sqrtf(g.t) * (g.i * rx[j].get(i));
        const float h = fmaf(g.a, total[i].h, in[j][i]);
        total[i] = Carry{begins ? -0.f : total[i].a * g.a, begins ? in[j][i] : h};
      }
    }

  // the waves' totals; before = what the waves above do to the state, whole = the tile
#pragma unroll
  for (int i = 0; i < V; ++i) totals[wave][lane * V + i] = total[i];
  lds_barrier();
  Carry before[V];
#pragma unroll
  for (int i = 0; i < V; ++i) before[i] = Carry{1.f, 0.f};
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int i = 0; i < V; ++i) before[i] = compose(before[i], totals[w][lane * V + i]);

  // the last wave has the tile's total, and gets the state before the tile
  const bool last = wave == kWaves - 1;
  Carry whole[V];
  const CarrySpace space = carry_space(a.work, tiles - 1, cols * a.b);
  uint64_t* words = space.words + (int64_t)column * 64 * V;
  uint32_t* flags = space.flags + (int64_t)column * (tiles - 1);
  const int64_t step = (int64_t)cols * a.b * 64 * V;
  uint64_t* mine = words + tile * step;  // and the lane's from lane * V
#pragma unroll
  for (int i = 0; i < V; ++i) whole[i] = compose(before[i], total[i]);
  if (last && tile > 0 && tile < tiles - 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) publish(mine + (uint32_t)(lane * V + i), whole[i]);
    if (lane == 0) raise_flag(flags + tile, 1);
  }
  float h[V];
  if (tile == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = a.h0 ? a.h0[(int64_t)b * a.c + chl + i] : 0.f;
  } else {
    look_back<V, kWaves>(words, step, flags, tile, wave, lane, last, gathered, h);
  }
  if (last) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float after = apply(whole[i], h[i]);
      if (tile < tiles - 1)
        publish(mine + (uint32_t)(lane * V + i), Carry{__uint_as_float(kWhole), after});
      else if (a.h_last && own)
        a.h_last[(int64_t)b * a.c + ch + i] = after;
      entry[lane * V + i] = h[i];
    }
    if (tile < tiles - 1 && lane == 0) raise_flag(flags + tile, 2);
  }
  lds_barrier();

#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = apply(before[i], entry[lane * V + i]);
  if (!own || n == 0) return;
  if (a.states && t0 % kEvery == 0) {
    const int pieces = (a.t + kEvery - 1) / kEvery;
#pragma unroll
    for (int i = 0; i < V; ++i)
      store_at(a.states + ((int64_t)b * pieces + t0 / kEvery) * a.c, (uint32_t)(ch + i) * 4, h[i]);
  }
  T* y = (T*)a.y + ((int64_t)b * a.t + t0) * a.c;
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < n) {
      P v;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[i] = STARTS && (first >> j & 1) ? in[j][i] : fmaf(av[j][i], h[i], in[j][i]);
        v.set(i, h[i]);
      }
      store_at(y + (int64_t)j * a.c, offset, v);
    }
}

// No rows: the state passes through.
__global__ __launch_bounds__(256) void scan_pass_kernel(const float* h0, int64_t n, float* h_last) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) h_last[i] = h0 ? h0[i] : 0.f;
}

int tiles_of(int t) { return (t + kTile - 1) / kTile; }

template <typename T, int V, bool STARTS, bool KEEP>
hipError_t run(const ScanArgs& a, hipStream_t s) {
  const int cols = (a.c + 64 * V - 1) / (64 * V), tiles = tiles_of(a.t);
  if (tiles > 1) {
    const hipError_t e = carry_clear(a.work, carry_bytes(tiles - 1, (int64_t)cols * a.b, 64 * V), s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((seq_scan_fwd_kernel<T, V, STARTS, KEEP>), dim3((unsigned)(cols * a.b * tiles)),
                     dim3(kWaves * 64), 0, s, a, cols, tiles);
  return hipGetLastError();
}
template <typename T, int V>
hipError_t run_as(const ScanArgs& a, hipStream_t s) {
  if (a.starts) return a.kept[0].q ? run<T, V, true, true>(a, s) : run<T, V, true, false>(a, s);
  return a.kept[0].q ? run<T, V, false, true>(a, s) : run<T, V, false, false>(a, s);
}
template <typename T>
hipError_t run_16(const ScanArgs& a, hipStream_t s) {
  const bool wide = a.c % 2 == 0 && pieces(a.x, 4, 2) && pieces(a.r, 4, 2) && pieces(a.i, 4, 2) && (uintptr_t)a.y % 4 == 0 &&
                    ((uintptr_t)a.kept[0].e | (uintptr_t)a.kept[1].e | (uintptr_t)a.kept[2].e) % 2 == 0;
  return wide ? run_as<T, 2>(a, s) : run_as<T, 1>(a, s);
}

}  // namespace

// For whichever of the two column widths needs more.
int64_t scan_fwd_work_bytes(int b, int t, int c) {
  const int64_t tiles = tiles_of(t);
  if (tiles <= 1 || b == 0) return 0;
  const int64_t narrow = carry_bytes(tiles - 1, (int64_t)b * ((c + 63) / 64), 64);
  const int64_t wide = carry_bytes(tiles - 1, (int64_t)b * ((c + 127) / 128), 128);
  return narrow > wide ? narrow : wide;
}

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s) {
  if (a.t == 0) {
    const int64_t n = (int64_t)a.b * a.c;
    if (a.h_last)
      hipLaunchKernelGGL(scan_pass_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.h0, n, a.h_last);
    return hipGetLastError();
  }
  if (a.dtype == convfwd::kF32) return run_as<float, 1>(a, s);
  if (a.dtype == convfwd::kF16) return run_16<_Float16>(a, s);
  return run_16<__bf16>(a, s);
}

}  // namespace convseq
