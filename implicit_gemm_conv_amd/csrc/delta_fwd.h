// delta_fwd.h -- gated delta rule forward: a wave carries 16 columns of one head's
// state through the chunks; kReplay computes only x of one chunk from its kept state.
// Included by one source for each type.
#include "delta_device.h"

namespace convdelta {

namespace {

enum Mode { kForward, kReplay };

// Operands of a chunk in LDS.
template <typename T, int DK>
struct FwdLds {
  static constexpr int NP = InParts<T>::n;
  __bf16 k[NP * RowsAt<DK>::part], q[NP * RowsAt<DK>::part];
  char solve[kMatrix], read[kMatrix];
  float rows[4 * kChunk];
};

template <typename T, int DK, int NW, Mode MODE>
struct Forward {
  static constexpr int NP = InParts<T>::n, KS = DK / 32, DT = DK / 16, kT = NW * 64;
  typedef FwdLds<T, DK> Lds;

  const DeltaArgs& a;
  Lds& s;
  int lane, m, q4, b, h, bh, col;
  bool live;
  f32x4_t state[DT];

  __device__ __forceinline__ Forward(const DeltaArgs& a_, Lds& s_, int bh_, int cb) : a(a_), s(s_), bh(bh_) {
    lane = threadIdx.x % 64;
    m = lane % 16;
    q4 = lane / 16;
    b = bh / a.hv;
    h = bh % a.hv;
    col = (cb * NW + wave_id()) * 16 + m;
    live = col < a.dv;
  }

  __device__ __forceinline__ void load_state(const float* from) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = row_of(t, 4 * q4 + r);
        state[t][r] = from && live && d < a.dk ? from[(int64_t)d * a.dv + col] : 0.f;
      }
  }
  __device__ __forceinline__ void store_state(float* to) const {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = row_of(t, 4 * q4 + r);
        if (live && d < a.dk) to[(int64_t)d * a.dv + col] = state[t][r];
      }
  }

  // values of the lane's rows of v
  __device__ __forceinline__ void load_v(int c, f32x4_t (&v)[4]) const {
    const T* p = (const T*)a.v.p + b * a.v.sb + h * a.v.sh + col;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = c * kChunk + row_of(t, 4 * q4 + r);
        v[t][r] = live && row < a.t ? to_f32(p[(int64_t)row * a.v.st]) : 0.f;
      }
  }

  __device__ __forceinline__ f32x4_t row4(int which, int t) const {
    return *(const f32x4_t*)(s.rows + which * kChunk + row_of(t, 4 * q4));
  }

  // A operand: rows of tile t of a matrix of rows, step k
  __device__ __forceinline__ Parts<NP> rows_of(const __bf16* x, int t, int k) const {
    return natural<NP>(x + row_of(t, m) * RowsAt<DK>::stride + 32 * k + 8 * q4, RowsAt<DK>::part);
  }
  // A operand: columns of tile t as rows, rows 32 k .. as its depth
  __device__ __forceinline__ Parts<NP> cols_of(const __bf16* x, int t, int k) const {
    return transposed<NP>(x + (32 * k + 8 * q4 + m / 4) * RowsAt<DK>::stride + 32 * (t >> 1) + 8 * (m % 4) + 4 * (t & 1),
                          RowsAt<DK>::stride, RowsAt<DK>::part);
  }
  __device__ __forceinline__ Parts<kParts> matrix(const char* x, int f) const {
    Parts<kParts> r;
#pragma unroll
    for (int n = 0; n < kParts; ++n) r.p[n] = *(const bf168_t*)(x + (f * kParts + n) * kFrag + lane * 16);
    return r;
  }

  // One chunk, all of its rows (ROW false), or row `only` alone.
  template <bool ROW>
  __device__ __forceinline__ bool chunk(int c, const f32x4_t (&v)[4], int only) {
    f32x4_t ks[4], qs[4], u[4];
    {
      Parts<kParts> sp[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k) sp[k] = operand<kParts>(state[2 * k], state[2 * k + 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        ks[t] = qs[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          ks[t] = mma(rows_of(s.k, t, k), sp[k], ks[t]);
          if (MODE == kForward) qs[t] = mma(rows_of(s.q, t, k), sp[k], qs[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // r, then x in place
    f32x4_t x[4], br[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4_t enter = row4(ROW ? 3 : 0, t), beta = row4(2, t);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[t][r] = v[t][r] - times(enter[r], ks[t][r]);
        br[t][r] = beta[r] * x[t][r];
        if (ROW && row_of(t, 4 * q4 + r) != only) br[t][r] = 0.f;
      }
    }
    if (!ROW) {
      Parts<kParts> bp[2] = {operand<kParts>(br[0], br[1]), operand<kParts>(br[2], br[3])};
#pragma unroll
      for (int f = 0; f < kTri; ++f) {
        x[low_t(f)] = mma(matrix(s.solve, f), bp[low_s(f)], x[low_t(f)]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    bool bad = false;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4_t beta = row4(2, t);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        u[t][r] = ROW ? br[t][r] : beta[r] * x[t][r];
        bad = bad || !finite(u[t][r]);
      }
    }
    if (!ROW && __any(bad)) return false;
    if (MODE == kReplay) {
      float* to = a.w.x + ((int64_t)bh * a.chunks + c) * kChunk * a.dvp + col;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = row_of(t, 4 * q4 + r);
          if (col < a.dvp && (!ROW || row == only)) to[(int64_t)row * a.dvp] = x[t][r];
        }
      if (!ROW) return true;
    }
    if (MODE == kForward) {
      const Parts<kParts> up[2] = {operand<kParts>(u[0], u[1]), operand<kParts>(u[2], u[3])};
      f32x4_t o[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f32x4_t enter = row4(ROW ? 3 : 0, t);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[t][r] = times(enter[r], qs[t][r]);
      }
#pragma unroll
      for (int f = 0; f < kTri; ++f) {
        Parts<kParts> p = matrix(s.read, f);
        if (ROW) keep(p, 32 * low_s(f) + 8 * q4, only, only + 1);
        o[low_t(f)] = mma(p, up[low_s(f)], o[low_t(f)]);
        __builtin_amdgcn_sched_barrier(0);
      }
      T* y = (T*)a.y + (((int64_t)b * a.t + c * kChunk) * a.hv + h) * a.dv + col;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = row_of(t, 4 * q4 + r);
          if (live && c * kChunk + row < a.t && (!ROW || row == only))
            y[(int64_t)row * a.hv * a.dv] = from_f32<T>(a.scale * o[t][r]);
        }
    }
    // the state moves on
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4_t leave = row4(1, t);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!ROW) u[t][r] = times(leave[r], u[t][r]);
    }
    const Parts<kParts> up[2] = {operand<kParts>(u[0], u[1]), operand<kParts>(u[2], u[3])};
    const float stay = s.rows[ROW ? 3 * kChunk + only : kChunk - 1];
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      f32x4_t n;
#pragma unroll
      for (int r = 0; r < 4; ++r) n[r] = times(stay, state[t][r]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Parts<NP> kt = cols_of(s.k, t, k);
        if (ROW) keep(kt, 32 * k + 8 * q4, only, only + 1);
        n = mma(kt, up[k], n);
      }
      state[t] = n;
      __builtin_amdgcn_sched_barrier(0);
    }
    return true;
  }

  // A chunk in which something is not finite goes row by row, so that it reaches only what comes after it.
  __device__ __forceinline__ void whole(int c, const f32x4_t (&v)[4]) {
    if (chunk<false>(c, v, 0)) return;
    const int n = min(kChunk, a.t - c * kChunk);
#pragma clang loop unroll(disable)
    for (int i = 0; i < n; ++i) chunk<true>(c, v, i);
    if (MODE == kReplay && col < a.dvp)  // rows past T hold nothing
      for (int i = n + q4; i < kChunk; i += 4) a.w.x[(((int64_t)bh * a.chunks + c) * kChunk + i) * a.dvp + col] = 0.f;
  }
};

template <typename T, int DK, int NW>
__global__ __launch_bounds__(NW * 64) void delta_fwd_kernel(DeltaArgs a, int blocks) {
  typedef Forward<T, DK, NW, kForward> F;
  __shared__ __attribute__((aligned(16))) typename F::Lds s;
  int bh, cb;
  if (!head_of(a.b * a.hv, blocks, bh, cb)) return;
  F f(a, s, bh, cb);
  const int64_t size = (int64_t)a.dk * a.dv;
  f.load_state(a.h0 ? a.h0 + bh * size : nullptr);
  Rows64<T, DK, F::kT> k, q;
  Stretch<kMatrix, F::kT> solve, read;
  Stretch<4 * kChunk * 4, F::kT> rows;
  f32x4_t v[4], next[4];
  const auto fetch = [&](int c) {
    const int64_t at = chunk_index(a, bh, c);
    k.load(a.k, f.b, f.h / (a.hv / a.hk), c * kChunk, a.t, a.dk, a.vec);
    q.load(a.q, f.b, f.h / (a.hv / a.hk), c * kChunk, a.t, a.dk, a.vec);
    solve.load(a.w.solve + at * kMatrix);
    read.load(a.w.read + at * kMatrix);
    rows.load(a.w.rows + at * 4 * kChunk);
    f.load_v(c, next);
  };
  if (a.chunks > 0) fetch(0);
  for (int c = 0; c < a.chunks; ++c) {
    __syncthreads();
    k.put(s.k);
    q.put(s.q);
    solve.put(s.solve);
    read.put(s.read);
    rows.put(s.rows);
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = next[t];
    __syncthreads();
    if (c + 1 < a.chunks) fetch(c + 1);
    if (a.states) f.store_state(a.states + (((int64_t)f.b * a.chunks + c) * a.hv + f.h) * size);
    f.whole(c, v);
  }
  f.store_state(a.h_last + bh * size);
}

template <typename T, int DK, int NW>
__global__ __launch_bounds__(NW * 64) void delta_replay_kernel(DeltaArgs a, int blocks) {
  typedef Forward<T, DK, NW, kReplay> F;
  __shared__ __attribute__((aligned(16))) typename F::Lds s;
  const int cb = blockIdx.x % blocks, c = blockIdx.x / blocks % a.chunks, bh = blockIdx.x / blocks / a.chunks;
  F f(a, s, bh, cb);
  const int64_t at = chunk_index(a, bh, c);
  Rows64<T, DK, F::kT> k;
  Stretch<kMatrix, F::kT> solve;
  Stretch<4 * kChunk * 4, F::kT> rows;
  f32x4_t v[4];
  k.load(a.k, f.b, f.h / (a.hv / a.hk), c * kChunk, a.t, a.dk, a.vec);
  solve.load(a.w.solve + at * kMatrix);
  rows.load(a.w.rows + at * 4 * kChunk);
  f.load_v(c, v);
  f.load_state(a.states_in + (((int64_t)f.b * a.chunks + c) * a.hv + f.h) * a.dk * a.dv);
  k.put(s.k);
  solve.put(s.solve);
  rows.put(s.rows);
  __syncthreads();
  f.whole(c, v);
}

template <typename T, int DK, int NW>
hipError_t fwd(const DeltaArgs& a, hipStream_t s) {
  const int blocks = (a.dv + 16 * NW - 1) / (16 * NW);
  hipLaunchKernelGGL((delta_fwd_kernel<T, DK, NW>), dim3((a.b * a.hv + 7) / 8 * 8 * blocks), dim3(NW * 64), 0, s, a, blocks);
  return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t delta_fwd_of(const DeltaArgs& a, hipStream_t s) {
  return for_dk(a.dk, [&](auto dk) { return fwd<T, decltype(dk)::value, 4>(a, s); });
}

template <typename T>
hipError_t delta_replay_of(const DeltaArgs& a, hipStream_t s) {
  return for_dk(a.dk, [&](auto dk) {
    constexpr int NW = 4;
    const int blocks = (a.dvp + 16 * NW - 1) / (16 * NW);
    hipLaunchKernelGGL((delta_replay_kernel<T, decltype(dk)::value, NW>), dim3(a.b * a.hv * a.chunks * blocks), dim3(NW * 64), 0,
                       s, a, blocks);
    return hipGetLastError();
  });
}

}  // namespace convdelta
