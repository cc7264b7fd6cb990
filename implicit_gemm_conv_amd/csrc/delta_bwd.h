// delta_bwd.h -- gated delta rule, the backward recurrence: a workgroup carries 16
// or 32 columns of the gradient of one head's state back through the chunks.  With dS the
// gradient of the state after a chunk and dy that of y,
//
//   du = leave * (k dS) + scale * R^T dy,  z = du + H^T (beta du)
//   dv = beta z  (the gradient of r as well),  dbeta = z . x
//   dS <- enter_last * dS + q^T (scale * enter * dy) - k^T (enter * beta z)
//
// z and each chunk's dS are left for the gradients that add over all columns
// (delta_grad.h).  The steps between barriers are those of delta_fwd.h: (1) du, (2) z,
// (3) the state's gradient.  The waves of the first role go the way from state to state,
// those of the second bring q and
// dy, and R^T dy a chunk ahead.  Bound as the forward recurrence is; 4 sequences of 4096 rows, 16 heads
// of 128 x 128, bf16: 320 us in 32 columns a workgroup (in 16, R^T dy took 37 us more of 468 in the first
// role).  Included by one source for each type.
#include "delta_team.h"

namespace convdelta {

namespace {

constexpr int kReadLd = kChunk + 4;  // spreads the columns over the banks

template <typename T, int DK, int NC>
struct BwdLds {
  typedef Team<T, DK, NC> F;
  __bf16 k[F::NP * RowsAt<DK>::part], q[F::NP * RowsAt<DK>::part];
  __bf16 state[NC][kParts * F::State::part];
  __bf16 dy[2][NC][F::NP * F::Rows::part];  // of the chunk, and of the one it goes on to
  float ry[NC][16 * kReadLd];               // scale * R^T dy by columns
  __bf16 bd[NC][kParts * F::Rows::part], in[NC][kParts * F::Rows::part], out[NC][kParts * F::Rows::part];
  float step[kChunk];
  int bad[2];
};

template <typename T, int DK, int NC, bool FIRST>
struct Backward : Team<T, DK, NC> {
  typedef Team<T, DK, NC> F;
  typedef BwdLds<T, DK, NC> Lds;
  using F::a;
  using F::q4;
  using F::m;
  using F::wave;
  using F::row;
  static constexpr int NP = F::NP, KS = F::KS;
  typedef typename F::Rows Rows;

  struct Chunk {
    Raw8<T> rows[KS];      // of k, or of q
    Parts<kParts> mat[2];  // of H^T, or the next chunk's R^T
    f32x4_t enter, leave, beta;
    float stay;
    T dy[NC][4];           // second role, the next chunk's
  };

  Lds& s;
  f32x4_t state[NC];
  int turn = 0;

  __device__ __forceinline__ Backward(const DeltaArgs& a_, Lds& s_, int bh_, int cb) : F(a_, bh_, cb), s(s_) {}

  __device__ __forceinline__ void fetch_matrix(int c, Parts<kParts> (&to)[2]) const {
    F::template load_matrix<true>(FIRST ? a.w.solve_t : a.w.read_t, c, to);
  }
  __device__ __forceinline__ void fetch_gates(int c, Chunk& x) const {
    x.enter = F::load_gate(0, c);
    if (FIRST) x.leave = F::load_gate(1, c), x.beta = F::load_gate(2, c);
    x.stay = F::load_stay(c);
  }
  // dy of chunk c into LDS (second role)
  __device__ __forceinline__ void put_dy(int c, const Chunk& x, f32x4_t (&d)[NC]) const {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) d[n][i] = c * kChunk + row() + i < a.t ? to_f32(x.dy[n][i]) : 0.f;
      F::template put<NP, Rows>(s.dy[c & 1][n], row(), d[n]);
    }
  }
  // scale * R^T dy of chunk c (second role), from the rows [lo, hi) where masked
  __device__ __forceinline__ void put_read(int c, const Parts<kParts> (&read)[2], bool masked, int lo, int hi) const {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      f32x4_t ry = {0.f, 0.f, 0.f, 0.f}, more = ry;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (F::template has<true>(k)) {
          Parts<NP> d = F::template get<NP, Rows>(s.dy[c & 1][n], k);
          if (masked) keep(d, 32 * k + 8 * q4, lo, hi);
          (k ? more : ry) = mma(read[k], d, k ? more : ry);
        }
      *(f32x4_t*)(s.ry[n] + m * kReadLd + row()) = a.scale * (ry + more);
    }
  }

  // (1) and (2) for all rows, or (masked) the rows [lo, hi) of one sequence, into z; kd is k dS.
  __device__ __forceinline__ void solve(int c, Chunk& x, const f32x4_t (&kd)[NC], bool masked, int lo, int hi,
                                        f32x4_t (&z)[NC]) {
    if (masked) {
      __syncthreads();  // what is read of the sequence before
      if (FIRST) {
        fetch_matrix(c, x.mat);
#pragma unroll
        for (int k = 0; k < 2; ++k) keep(x.mat[k], 32 * k + 8 * q4, lo, hi);
      } else {
        Parts<kParts> read[2];
        fetch_matrix(c, read);
#pragma unroll
        for (int k = 0; k < 2; ++k) keep(read[k], 32 * k + 8 * q4, lo, hi);
        put_read(c, read, true, lo, hi);
      }
      wait_for_memory();
      __syncthreads();
    }
    f32x4_t du[NC], hd[NC], more[NC];  // sums of their own, added once (see delta_fwd.h)
    if (FIRST)
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        f32x4_t bd;
        const f32x4_t ry = *(const f32x4_t*)(s.ry[n] + m * kReadLd + row());
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool out = row() + i < lo || row() + i >= hi;
          du[n][i] = out ? 0.f : times(x.leave[i], kd[n][i]) + ry[i];
          bd[i] = out ? 0.f : x.beta[i] * du[n][i];
        }
        F::template put<kParts, Rows>(s.bd[n], row(), bd);
        hd[n] = more[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    __syncthreads();
    if (FIRST) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (F::template has<true>(k))
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const auto bp = F::template get<kParts, Rows>(s.bd[n], k);
            (k ? more : hd)[n] = mma(x.mat[k], bp, (k ? more : hd)[n]);
          }
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row() + i >= lo && row() + i < hi) z[n][i] = du[n][i] + (hd[n][i] + more[n][i]);
    }
  }

  __device__ __forceinline__ void chunk(int c, Chunk& x, f32x4_t (&dy)[NC]) {
    const int next = max(c - 1, 0), then = max(c - 2, 0);
    __syncthreads();  // the state's parts and dy are there
    F::put_rows(FIRST ? s.k : s.q, x.rows);
    f32x4_t kd[NC];
    if (FIRST) {
      f32x4_t more[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) kd[n] = more[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const Parts<NP> rows = F::rows_of(x.rows, k);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          f32x4_t& to = (k & 1 ? more : kd)[n];
          to = mma(rows, F::template get<kParts, typename F::State>(s.state[n], k), to);
        }
      }
#pragma unroll
      for (int n = 0; n < NC; ++n) kd[n] += more[n];
    } else {
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        f32x4_t in;
#pragma unroll
        for (int i = 0; i < 4; ++i) in[i] = times(x.enter[i], a.scale * dy[n][i]);
        F::template put<kParts, Rows>(s.in[n], row(), in);
      }
    }
    F::load_rows(FIRST ? a.k : a.q, next, x.rows);
    f32x4_t ahead[NC];
    if (!FIRST) {
      put_dy(next, x, ahead);
      F::load_col(a.dy, then, x.dy);
    }
    // All rows at once, and where something is not finite once more, each sequence by itself, so that nothing crosses a
    // start.  `first`: the rows that the state before the chunk reaches are those of the first sequence.
    f32x4_t z[NC];
    bool masked = false;
    int first = kChunk;
#pragma clang loop unroll(disable)
    for (;;) {
      int hi = kChunk;
#pragma clang loop unroll(disable)
      do {
        int lo = 0;
        if (masked) {
          lo = hi - 1;
          while (lo > 0 && s.step[lo] != 0.f) --lo;
          if (lo > 0 || s.step[0] == 0.f) first = lo;
        }
        solve(c, x, kd, masked, lo, hi, z);
        hi = lo;
      } while (hi > 0);
      if (FIRST) {
        float test = 0.f;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          f32x4_t out;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            test = fmaf(z[n][i], 0.f, test);
            if (c * kChunk + row() + i >= a.t) z[n][i] = 0.f;  // rows past T hold nothing, whatever the state's gradient is
            out[i] = -times(x.enter[i], x.beta[i] * z[n][i]);
          }
          F::template put<kParts, Rows>(s.out[n], row(), out);
        }
        if (__any(test != 0.f)) s.bad[turn & 1] = 1;  // NaN
      }
      __syncthreads();
      const bool bad = s.bad[turn & 1];
      if (threadIdx.x == 0) s.bad[~turn & 1] = 0;
      ++turn;
      if (masked || !bad) break;
      masked = true;
      if (threadIdx.x < kChunk) s.step[threadIdx.x] = a.w.rows[(chunk_index(a, F::bh, c) * 4 + 3) * kChunk + threadIdx.x];
      wait_for_memory();
      __syncthreads();
    }
    if (FIRST) {
      fetch_matrix(next, x.mat);
    } else {
      put_read(next, x.mat, false, 0, kChunk);
      fetch_matrix(then, x.mat);
    }
    // (3), from the rows [0, first) where masked
    if (F::has_tile()) {
      f32x4_t qi[NC], more[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) qi[n] = more[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Parts<NP> qt = F::cols_of(s.q, F::tile, k), kt = F::cols_of(s.k, F::tile, k);
        if (masked) keep(qt, 32 * k + 8 * q4, 0, first), keep(kt, 32 * k + 8 * q4, 0, first);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          qi[n] = mma(qt, F::template get<kParts, Rows>(s.in[n], k), qi[n]);
          more[n] = mma(kt, F::template get<kParts, Rows>(s.out[n], k), more[n]);
        }
      }
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) state[n][i] = times(x.stay, state[n][i]) + (qi[n][i] + more[n][i]);
      F::put_state(s.state, state);
    }
    // stores come after the loads of the next chunk (see delta_fwd.h)
    if (FIRST) {
      const Range zs(a.w.z + chunk_index(a, F::bh, c) * kChunk * a.dvp, (int64_t)kChunk * a.dvp * 4);
      f32x4_t dx[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dx[n][i] = x.beta[i] * z[n][i];
          if (F::col(n) >= a.dv) z[n][i] = 0.f;
        }
      fetch_gates(next, x);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const uint32_t at = F::col(n) < a.dvp ? (uint32_t)(row() * a.dvp + F::col(n)) * 4u : kNowhere;
#pragma unroll
        for (int i = 0; i < 4; ++i) zs.store(at + (uint32_t)(i * a.dvp) * 4u, z[n][i]);
      }
      F::template store_col<T>(a.dv_, c, dx);
    } else {
      fetch_gates(next, x);
#pragma unroll
      for (int n = 0; n < NC; ++n) dy[n] = ahead[n];
    }
    keep_state(c - 1);
  }
  // The gradient of the state after chunk c.
  __device__ __forceinline__ void keep_state(int c) const {
    F::store_state(c >= 0 ? a.w.dstate + chunk_index(a, F::bh, c) * a.dk * a.dvp : nullptr, a.dvp, a.dvp, state);
  }

  __device__ __forceinline__ void run() {
    const int64_t size = (int64_t)a.dk * a.dv;
    F::load_state(a.dh_last ? a.dh_last + F::bh * size : nullptr, state);
    F::put_state(s.state, state);
    if (a.chunks > 0) {
      Chunk x;
      const int last = a.chunks - 1, next = max(last - 1, 0);
      f32x4_t dy[NC];
      if (!FIRST) {
        F::load_col(a.dy, last, x.dy);
        put_dy(last, x, dy);
      }
      fetch_matrix(last, x.mat);
      __syncthreads();
      if (!FIRST) {
        put_read(last, x.mat, false, 0, kChunk);
        fetch_matrix(next, x.mat);
        F::load_col(a.dy, next, x.dy);
      }
      F::load_rows(FIRST ? a.k : a.q, last, x.rows);
      fetch_gates(last, x);
      keep_state(last);
      for (int c = last; c >= 0; --c) chunk(c, x, dy);
    }
    F::store_state(a.dh0 + F::bh * size, a.dv, a.dv, state);
  }
};

template <typename T, int DK, int NC>
__global__ __launch_bounds__(kTeam, 2) void delta_bwd_kernel(DeltaArgs a, int blocks) {
  __shared__ __attribute__((aligned(16))) BwdLds<T, DK, NC> s;
  int bh, cb;
  if (!head_of(a.b * a.hv, blocks, bh, cb)) return;
  if (threadIdx.x < 2) s.bad[threadIdx.x] = 0;
  if (wave_id() < 4)
    Backward<T, DK, NC, true>(a, s, bh, cb).run();
  else
    Backward<T, DK, NC, false>(a, s, bh, cb).run();
}

}  // namespace

template <typename T>
hipError_t delta_bwd_of(const DeltaArgs& a, hipStream_t s) {
  return for_dk(a.dk, [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    return for_columns(a, [&](auto nc) {
      // two tiles need more LDS than there is with the widest heads in fp32 and fp16 (there by 776 bytes: 4096 rows, 64 heads
      // of 128 x 128, both take 16 columns, the backward pass 1074 us where bf16 has 836)
      constexpr int NC = sizeof(BwdLds<T, DK, decltype(nc)::value>) <= 160 * 1024 ? decltype(nc)::value : 1;
      const int blocks = a.dvp / (16 * NC);
      hipLaunchKernelGGL((delta_bwd_kernel<T, DK, NC>), dim3((a.b * a.hv + 7) / 8 * 8 * blocks), dim3(kTeam), 0, s, a, blocks);
      return hipGetLastError();
    });
  });
}

}  // namespace convdelta
