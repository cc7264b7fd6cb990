// delta_bwd.h -- gated delta rule, the backward recurrence: a wave carries 16 columns
// of the gradient of one head's state back through the chunks.  With dS the gradient
// of the state after a chunk and dy that of y,
//
//   du = leave * (k dS) + scale * R^T dy,  z = du + H^T (beta du)
//   dv = beta z  (the gradient of r as well),  dbeta = z . x
//   dS <- enter_last * dS + q^T (scale * enter * dy) - k^T (enter * beta z)
//
// z and each chunk's dS are left for the gradients that add over all columns
// (delta_grad.h).  Included by one source for each type.
#include "delta_device.h"

namespace convdelta {

namespace {

template <typename T, int DK>
struct BwdLds {
  static constexpr int NP = InParts<T>::n;
  __bf16 k[NP * RowsAt<DK>::part], q[NP * RowsAt<DK>::part];
  char solve[kMatrix], read[kMatrix];
  float rows[4 * kChunk];
};

template <typename T, int DK, int NW>
struct Backward {
  static constexpr int NP = InParts<T>::n, KS = DK / 32, DT = DK / 16, kT = NW * 64;
  typedef BwdLds<T, DK> Lds;

  const DeltaArgs& a;
  Lds& s;
  int lane, m, q4, b, h, bh, col;
  bool live;
  f32x4_t state[DT];

  __device__ __forceinline__ Backward(const DeltaArgs& a_, Lds& s_, int bh_, int cb) : a(a_), s(s_), bh(bh_) {
    lane = threadIdx.x % 64;
    m = lane % 16;
    q4 = lane / 16;
    b = bh / a.hv;
    h = bh % a.hv;
    col = (cb * NW + wave_id()) * 16 + m;
    live = col < a.dv;
  }

  __device__ __forceinline__ void load_dy(int c, f32x4_t (&v)[4]) const {
    const T* p = (const T*)a.dy.p + b * a.dy.sb + h * a.dy.sh + col;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = c * kChunk + row_of(t, 4 * q4 + r);
        v[t][r] = live && row < a.t ? to_f32(p[(int64_t)row * a.dy.st]) : 0.f;
      }
  }
  __device__ __forceinline__ f32x4_t row4(int which, int t) const {
    return *(const f32x4_t*)(s.rows + which * kChunk + row_of(t, 4 * q4));
  }
  __device__ __forceinline__ Parts<NP> rows_of(const __bf16* x, int t, int k) const {
    return natural<NP>(x + row_of(t, m) * RowsAt<DK>::stride + 32 * k + 8 * q4, RowsAt<DK>::part);
  }
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

  // z of the rows [lo, hi) (MASKED), or of all; whether they are finite.
  template <bool MASKED>
  __device__ __forceinline__ bool solve(const f32x4_t (&kd)[4], const Parts<NP> (&dp)[2], f32x4_t (&z)[4], int lo, int hi) {
    f32x4_t du[4], bd[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) du[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int f = 0; f < kTri; ++f) {
      Parts<kParts> p = matrix(s.read, f);
      Parts<NP> d = dp[up_s(f)];
      if (MASKED) keep(p, 32 * up_s(f) + 8 * q4, lo, hi), keep(d, 32 * up_s(f) + 8 * q4, lo, hi);
      du[up_t(f)] = mma(p, d, du[up_t(f)]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4_t leave = row4(1, t), beta = row4(2, t);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row_of(t, 4 * q4 + r);
        du[t][r] = times(leave[r], kd[t][r]) + a.scale * du[t][r];
        const bool out = MASKED && (row < lo || row >= hi);
        if (out) du[t][r] = 0.f;
        bd[t][r] = out ? 0.f : beta[r] * du[t][r];
      }
    }
    const Parts<kParts> bp[2] = {operand<kParts>(bd[0], bd[1]), operand<kParts>(bd[2], bd[3])};
#pragma unroll
    for (int f = 0; f < kTri; ++f) {
      Parts<kParts> p = matrix(s.solve, f);
      if (MASKED) keep(p, 32 * up_s(f) + 8 * q4, lo, hi);
      du[up_t(f)] = mma(p, bp[up_s(f)], du[up_t(f)]);
      __builtin_amdgcn_sched_barrier(0);
    }
    bool bad = false;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row_of(t, 4 * q4 + r);
        bad = bad || !finite(du[t][r]);
        if (!MASKED || (row >= lo && row < hi)) z[t][r] = du[t][r];
      }
    return !__any(bad);
  }

  __device__ __forceinline__ void chunk(int c, const f32x4_t (&dy)[4]) {
    f32x4_t kd[4], z[4];
    {
      Parts<kParts> sp[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k) sp[k] = operand<kParts>(state[2 * k], state[2 * k + 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        kd[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) kd[t] = mma(rows_of(s.k, t, k), sp[k], kd[t]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    const Parts<NP> dp[2] = {operand<NP>(dy[0], dy[1]), operand<NP>(dy[2], dy[3])};
    // rows that the state before the chunk reaches: all, or those of the first sequence
    int first = kChunk;
    const bool masked = !solve<false>(kd, dp, z, 0, kChunk);
    if (masked) {
      // something is not finite: each sequence by itself, so that nothing crosses a start
      int hi = kChunk;
#pragma clang loop unroll(disable)
      for (int lo = kChunk - 1; lo >= 0; --lo)
        if (lo == 0 || s.rows[3 * kChunk + lo] == 0.f) {
          solve<true>(kd, dp, z, lo, hi);
          hi = lo;
          if (lo > 0 || s.rows[3 * kChunk] == 0.f) first = lo;
        }
    }
    f32x4_t in[4], out[4];
    T* dv = (T*)a.dv_ + (((int64_t)b * a.t + c * kChunk) * a.hv + h) * a.dv + col;
    float* zs = a.w.z + ((int64_t)bh * a.chunks + c) * kChunk * a.dvp + col;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4_t enter = row4(0, t), beta = row4(2, t);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row_of(t, 4 * q4 + r);
        if (c * kChunk + row >= a.t) z[t][r] = 0.f;  // rows past T hold nothing, whatever the state's gradient is
        const float dx = beta[r] * z[t][r];
        if (live && c * kChunk + row < a.t) dv[(int64_t)row * a.hv * a.dv] = from_f32<T>(dx);
        if (col < a.dvp) zs[(int64_t)row * a.dvp] = z[t][r];
        in[t][r] = times(enter[r], a.scale * dy[t][r]);
        out[t][r] = -times(enter[r], dx);
      }
    }
    const Parts<kParts> ip[2] = {operand<kParts>(in[0], in[1]), operand<kParts>(in[2], in[3])};
    const Parts<kParts> op[2] = {operand<kParts>(out[0], out[1]), operand<kParts>(out[2], out[3])};
    const float stay = s.rows[kChunk - 1];
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      f32x4_t n;
#pragma unroll
      for (int r = 0; r < 4; ++r) n[r] = times(stay, state[t][r]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Parts<NP> qt = cols_of(s.q, t, k), kt = cols_of(s.k, t, k);
        if (masked) keep(qt, 32 * k + 8 * q4, 0, first), keep(kt, 32 * k + 8 * q4, 0, first);
        n = mma(qt, ip[k], n);
        n = mma(kt, op[k], n);
      }
      state[t] = n;
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

template <typename T, int DK, int NW>
__global__ __launch_bounds__(NW * 64) void delta_bwd_kernel(DeltaArgs a, int blocks) {
  typedef Backward<T, DK, NW> F;
  __shared__ __attribute__((aligned(16))) typename F::Lds s;
  int bh, cb;
  if (!head_of(a.b * a.hv, blocks, bh, cb)) return;
  F f(a, s, bh, cb);
  const int64_t size = (int64_t)a.dk * a.dv;
#pragma unroll
  for (int t = 0; t < F::DT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = row_of(t, 4 * f.q4 + r);
      f.state[t][r] = a.dh_last && f.live && d < a.dk ? a.dh_last[bh * size + (int64_t)d * a.dv + f.col] : 0.f;
    }
  Rows64<T, DK, F::kT> k, q;
  Stretch<kMatrix, F::kT> solve, read;
  Stretch<4 * kChunk * 4, F::kT> rows;
  f32x4_t dy[4], next[4];
  const auto fetch = [&](int c) {
    const int64_t at = chunk_index(a, bh, c);
    k.load(a.k, f.b, f.h / (a.hv / a.hk), c * kChunk, a.t, a.dk, a.vec);
    q.load(a.q, f.b, f.h / (a.hv / a.hk), c * kChunk, a.t, a.dk, a.vec);
    solve.load(a.w.solve_t + at * kMatrix);
    read.load(a.w.read_t + at * kMatrix);
    rows.load(a.w.rows + at * 4 * kChunk);
    f.load_dy(c, next);
  };
  if (a.chunks > 0) fetch(a.chunks - 1);
  for (int c = a.chunks - 1; c >= 0; --c) {
    __syncthreads();
    k.put(s.k);
    q.put(s.q);
    solve.put(s.solve);
    read.put(s.read);
    rows.put(s.rows);
#pragma unroll
    for (int t = 0; t < 4; ++t) dy[t] = next[t];
    __syncthreads();
    if (c > 0) fetch(c - 1);
    float* ds = a.w.dstate + chunk_index(a, bh, c) * a.dk * a.dvp + f.col;
#pragma unroll
    for (int t = 0; t < F::DT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = row_of(t, 4 * f.q4 + r);
        if (f.col < a.dvp && d < a.dk) ds[(int64_t)d * a.dvp] = f.state[t][r];
      }
    f.chunk(c, dy);
  }
#pragma unroll
  for (int t = 0; t < F::DT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = row_of(t, 4 * f.q4 + r);
      if (f.live && d < a.dk) a.dh0[bh * size + (int64_t)d * a.dv + f.col] = f.state[t][r];
    }
}

}  // namespace

template <typename T>
hipError_t delta_bwd_of(const DeltaArgs& a, hipStream_t s) {
  return for_dk(a.dk, [&](auto dk) {
    constexpr int NW = 4;
    const int blocks = (a.dvp + 16 * NW - 1) / (16 * NW);
    hipLaunchKernelGGL((delta_bwd_kernel<T, decltype(dk)::value, NW>), dim3((a.b * a.hv + 7) / 8 * 8 * blocks), dim3(NW * 64), 0,
                       s, a, blocks);
    return hipGetLastError();
  });
}

}  // namespace convdelta
