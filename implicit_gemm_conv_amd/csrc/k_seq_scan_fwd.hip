// k_seq_scan_fwd.hip -- gated linear recurrence, forward, in one pass over the
// inputs.
//
//   r = sigmoid(gate_r), i = sigmoid(gate_i), u = decay * softplus(lam) * r, a = e^-u
//   h_t = a_t h_{t-1} + sqrt(1 - a^2) i x_t
//
// A workgroup of 8 waves takes a tile of 128 rows by 64 channels, a wave 16 rows
// of it, a lane one channel of those.  The lane composes its rows into one step
// h -> A h + H, the waves' steps are composed through LDS, the tiles' through
// memory (seq_carry.h), and with the state before its rows known the lane runs
// the recurrence over the a and m i x it still holds.  Each input is read once
// and y written once: memory bound, 4 elements a value.
//
// 1x65539x1024 bf16 takes 124 us (4.3 TB/s, where a copy reaches 5.1), 4x4096x2048
// with 8 bits kept 95 to 104 us, the vector ALU busy 60% of it.  One channel a lane: its
// registers let four workgroups (three with 8 bits) share a compute unit and cover
// each other's waits; three for four costs 9% at 4x4096x2048 without 8 bits (69 us
// for 64 back to back) and 1 to 2% on the long sequence.  Tiles of 64 rows take 190 us
// on the one long sequence, which has twice the tiles to look back over, and 96 on the
// other, where 128 take 99 to 102.
#include "seq_carry.h"

namespace convseq {

namespace {

constexpr int kWaves = 8;
constexpr int kTile = kWaves * kGroup;  // rows

template <typename T, bool STARTS, bool KEEP>
__global__ __launch_bounds__(kWaves * 64, KEEP ? 6 : 8) void seq_scan_fwd_kernel(ScanArgs a, int cols, int tiles) {
  __shared__ Carry totals[kWaves][64];
  __shared__ float entry[64], rates[64];
  __shared__ Gathered<1, kWaves> gathered;
  __shared__ int ticket;
  typedef Pack<T, 1> P;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // turned by one a tile row: each column's tiles go to all 8 dies, not to one of
  // them (1x65539x1024 bf16: 125 us instead of 193)
  const int columns = cols * a.b, column = (blockIdx.x + blockIdx.x / columns) % columns;
  const int tile = tiles > 1 ? take_ticket(a.work, column, &ticket) : 0;
  const int b = column / cols;
  const int ch = column % cols * 64 + lane;
  const int chl = min(ch, a.c - 1);  // lanes past the last channel read it again
  const bool own = ch < a.c;
  const int t0 = tile * kTile + wave * kGroup;
  const int n = min(max(a.t - t0, 0), kGroup);  // rows of this wave

  // rows past the last read it again
  const int64_t row = min(t0, a.t - 1);
  const auto walk = [&](const Rows& r) {
    return RowWalk((const T*)r.p + b * r.sb + row * r.st, r.st * (int64_t)sizeof(T));
  };
  P rx[kGroup], rr[kGroup], ri[kGroup];
  {
    uint32_t offset = (uint32_t)chl * sizeof(T);
    renew(offset);
    RowWalk wx = walk(a.x), wr = walk(a.r), wi = walk(a.i);
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      rx[j] = wx.load<P>(offset);
      rr[j] = wr.load<P>(offset);
      ri[j] = wi.load<P>(offset);
      wx.step(j + 1 < n);
      wr.step(j + 1 < n);
      wi.step(j + 1 < n);
    }
  }
  uint32_t first = 0;  // bit j: row t0 + j begins a sequence
  if (STARTS) first = (uint32_t)__ballot(lane < n && a.starts[(int64_t)b * a.t + t0 + lane]);
  if (wave == 0) rates[lane] = a.decay * softplus(a.lam[chl]);
  lds_barrier();
  const Rate rate = rate_of(rates[lane]);

  if (KEEP && n > 0 && own) {
    const int64_t at = (int64_t)b * ((a.t + kGroup - 1) / kGroup) + t0 / kGroup;
    keep_group<T, 1>(rx, n, a.kept[0], at, a.c, ch);
    keep_group<T, 1>(rr, n, a.kept[1], at, a.c, ch);
    keep_group<T, 1>(ri, n, a.kept[2], at, a.c, ch);
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      renew(rx[j]);
      renew(rr[j]);
      renew(ri[j]);
    }
  }

  float av[kGroup], in[kGroup];  // a and m i x
  Carry total = {1.f, 0.f};
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < n) {
      const bool begins = STARTS && (first >> j & 1);
      const Gate g = gates(-kLog2e * rr[j].get(0), -kLog2e * ri[j].get(0), rate);
      av[j] = g.a;
      in[j] = __builtin_amdgcn_sqrtf(g.t) * (g.i * rx[j].get(0));
      const float h = fmaf(g.a, total.h, in[j]);
      total = Carry{begins ? -0.f : total.a * g.a, begins ? in[j] : h};
    }

  total.a = positive(total.a);

  // the waves' totals; before = what the waves above do to the state
  totals[wave][lane] = total;
  lds_barrier();
  Carry before = {1.f, 0.f};
  for (int w = 0; w < wave; ++w) before = compose(before, totals[w][lane]);

  // the last wave has the tile's total, and gets the state before the tile
  const bool last = wave == kWaves - 1;
  const Carry whole = compose(before, total);
  const CarrySpace space = carry_space(a.work, tiles - 1, columns);
  const int64_t step = (int64_t)columns * 64;
  uint64_t* words = space.words + (int64_t)column * 64;
  uint64_t* mine = words + tile * step;  // and the lane's from lane
  uint32_t* flags = space.flags + (int64_t)column * (tiles - 1);
  if (last && tile > 0 && tile < tiles - 1) {
    publish(mine + (uint32_t)lane, whole);
    if (lane == 0) raise_flag(flags + tile, 1);
  }
  float state[1];
  if (tile == 0)
    state[0] = a.h0 ? a.h0[(int64_t)b * a.c + chl] : 0.f;
  else
    look_back<1, kWaves>(words, step, flags, tile, wave, lane, last, gathered, state);
  if (last) {
    const float after = apply(whole, state[0]);
    if (tile < tiles - 1) {
      publish(mine + (uint32_t)lane, Carry{__uint_as_float(kWhole), after});
      if (lane == 0) raise_flag(flags + tile, 2);
    } else if (a.h_last && own) {
      a.h_last[(int64_t)b * a.c + ch] = after;
    }
    entry[lane] = state[0];
  }
  lds_barrier();

  float h = apply(before, entry[lane]);
  if (!own || n == 0) return;
  if (a.states && t0 % kEvery == 0) {
    const int pieces = (a.t + kEvery - 1) / kEvery;
    store_at(a.states + ((int64_t)b * pieces + t0 / kEvery) * a.c, (uint32_t)ch * 4, h);
  }
  const auto store_rows = [&](auto whole) {
    uint32_t offset = (uint32_t)ch * sizeof(T);
    renew(offset);
    RowWalk y((T*)a.y + ((int64_t)b * a.t + t0) * a.c, (int64_t)a.c * sizeof(T));
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (decltype(whole)::value || j < n) {
        h = STARTS && (first >> j & 1) ? in[j] : fmaf(av[j], h, in[j]);
        P v;
        v.set(0, h);
        y.store(offset, v);
        y.step();
      }
  };
  if (n == kGroup)
    store_rows(Yes{});
  else
    store_rows(No{});
}

// No rows: the state passes through.
__global__ __launch_bounds__(256) void scan_pass_kernel(const float* h0, int64_t n, float* h_last) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) h_last[i] = h0 ? h0[i] : 0.f;
}

int tiles_of(int t) { return (t + kTile - 1) / kTile; }
int cols_of(int c) { return (c + 63) / 64; }

template <typename T, bool STARTS, bool KEEP>
hipError_t run(const ScanArgs& a, hipStream_t s) {
  const int cols = cols_of(a.c), tiles = tiles_of(a.t);
  if (tiles > 1) {
    const hipError_t e = carry_clear(a.work, carry_bytes(tiles - 1, (int64_t)cols * a.b, 64), s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((seq_scan_fwd_kernel<T, STARTS, KEEP>), dim3((unsigned)(cols * a.b * tiles)), dim3(kWaves * 64), 0,
                     s, a, cols, tiles);
  return hipGetLastError();
}
template <typename T>
hipError_t run_as(const ScanArgs& a, hipStream_t s) {
  if (a.starts) return a.kept[0].q ? run<T, true, true>(a, s) : run<T, true, false>(a, s);
  return a.kept[0].q ? run<T, false, true>(a, s) : run<T, false, false>(a, s);
}

}  // namespace

int64_t scan_fwd_work_bytes(int b, int t, int c) {
  const int64_t tiles = tiles_of(t);
  return tiles > 1 && b > 0 ? carry_bytes(tiles - 1, (int64_t)b * cols_of(c), 64) : 0;
}

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s) {
  if (a.t == 0) {
    const int64_t n = (int64_t)a.b * a.c;
    if (a.h_last)
      hipLaunchKernelGGL(scan_pass_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.h0, n, a.h_last);
    return hipGetLastError();
  }
  if (a.dtype == convfwd::kF32) return run_as<float>(a, s);
  if (a.dtype == convfwd::kF16) return run_as<_Float16>(a, s);
  return run_as<__bf16>(a, s);
}

}  // namespace convseq
