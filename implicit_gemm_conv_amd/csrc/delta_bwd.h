// delta_bwd.h -- gated delta rule, the backward recurrence: a workgroup carries 16
// columns of the gradient of one head's state back through the chunks.  With dS the
// gradient of the state after a chunk and dy that of y,
//
//   du = leave * (k dS) + scale * R^T dy,  z = du + H^T (beta du)
//   dv = beta z  (the gradient of r as well),  dbeta = z . x
//   dS <- enter_last * dS + q^T (scale * enter * dy) - k^T (enter * beta z)
//
// z and each chunk's dS are left for the gradients that add over all columns
// (delta_grad.h).  The steps between barriers are those of delta_fwd.h: (1) du, (2) z,
// (3) the state's gradient.  Included by one source for each type.
#include "delta_team.h"

namespace convdelta {

namespace {

template <typename T, int DK>
struct BwdLds {
  typedef Team<T, DK> F;
  __bf16 k[F::NP * RowsAt<DK>::part], q[F::NP * RowsAt<DK>::part];
  __bf16 state[kParts * F::State::part];
  __bf16 dy[F::NP * F::Rows::part], bd[kParts * F::Rows::part], in[kParts * F::Rows::part], out[kParts * F::Rows::part];
  float step[kChunk];
  int bad[2];
};

template <typename T, int DK>
struct Backward : Team<T, DK> {
  typedef Team<T, DK> F;
  typedef BwdLds<T, DK> Lds;
  using F::a;
  using F::q4;
  using F::m;
  using F::wave;
  using F::col;
  using F::row;
  static constexpr int NP = F::NP, KS = F::KS;

  struct Chunk {
    Raw8<T> k[KS], q[KS];
    Parts<kParts> solve[2], read[2];
    Gates g;
    T dy[4];
  };

  Lds& s;
  f32x4_t state[F::own];
  int turn = 0;

  __device__ __forceinline__ Backward(const DeltaArgs& a_, Lds& s_, int bh_, int cb) : F(a_, bh_, cb), s(s_) {}

  __device__ __forceinline__ void fetch_rows(int c, Chunk& x) const {
    F::load_rows(a.k, c, x.k);
    F::load_rows(a.q, c, x.q);
    F::load_col(a.dy, c, x.dy);
  }
  __device__ __forceinline__ void fetch(int c, Chunk& x) const {
    fetch_rows(c, x);
    F::template load_matrix<true>(a.w.solve_t, c, x.solve);
    F::template load_matrix<true>(a.w.read_t, c, x.read);
    x.g = F::load_gates(c);
  }
  __device__ __forceinline__ f32x4_t dy_of(int c, const Chunk& x) const {
    f32x4_t d;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = c * kChunk + row() + i < a.t ? to_f32(x.dy[i]) : 0.f;
    return d;
  }

  // (1) and (2) for all rows, or (masked) the rows [lo, hi) of one sequence, into z; kd is k dS.
  __device__ __forceinline__ void solve(int c, Chunk& x, const f32x4_t& kd, bool masked, int lo, int hi, f32x4_t& z) {
    if (masked) {
      F::template load_matrix<true>(a.w.solve_t, c, x.solve);
      F::template load_matrix<true>(a.w.read_t, c, x.read);
#pragma unroll
      for (int k = 0; k < 2; ++k) keep(x.solve[k], 32 * k + 8 * q4, lo, hi), keep(x.read[k], 32 * k + 8 * q4, lo, hi);
      wait_for_memory();
    }
    f32x4_t ry = {0.f, 0.f, 0.f, 0.f}, more = ry;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (F::template has<true>(k)) {
        Parts<NP> d = F::template get<NP, typename F::Rows>(s.dy, k);
        if (masked) keep(d, 32 * k + 8 * q4, lo, hi);
        (k ? more : ry) = mma(x.read[k], d, k ? more : ry);
      }
    f32x4_t du, bd;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool out = row() + i < lo || row() + i >= hi;
      du[i] = out ? 0.f : times(x.g.leave[i], kd[i]) + a.scale * (ry[i] + more[i]);
      bd[i] = out ? 0.f : x.g.beta[i] * du[i];
    }
    if (masked) __syncthreads();  // what is read of the sequence before
    F::template put<kParts, typename F::Rows>(s.bd, row(), bd);
    __syncthreads();
    more = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (F::template has<true>(k)) {
        const auto bp = F::template get<kParts, typename F::Rows>(s.bd, k);
        (k ? more : du) = mma(x.solve[k], bp, k ? more : du);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row() + i >= lo && row() + i < hi) z[i] = du[i] + more[i];
  }

  // What a wave gives to (3).
  __device__ __forceinline__ void give(int c, const Chunk& x, f32x4_t& z, const f32x4_t& dy) {
    f32x4_t in, out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c * kChunk + row() + i >= a.t) z[i] = 0.f;  // rows past T hold nothing, whatever the state's gradient is
      in[i] = times(x.g.enter[i], a.scale * dy[i]);
      out[i] = -times(x.g.enter[i], x.g.beta[i] * z[i]);
    }
    F::template put<kParts, typename F::Rows>(s.in, row(), in);
    F::template put<kParts, typename F::Rows>(s.out, row(), out);
  }
  __device__ __forceinline__ void store(int c, const f32x4_t& beta, const f32x4_t& z) const {
    const Range zs(a.w.z + chunk_index(a, F::bh, c) * kChunk * a.dvp, (int64_t)kChunk * a.dvp * 4);
    const uint32_t at = col < a.dvp ? (uint32_t)(row() * a.dvp + col) * 4u : kNowhere;
    f32x4_t dx;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dx[i] = beta[i] * z[i];
      zs.store(at + (uint32_t)(i * a.dvp) * 4u, F::live ? z[i] : 0.f);
    }
    F::store_col(a.dv_, c, dx);
  }
  // (3), from the rows [0, first) where masked
  __device__ __forceinline__ void move(float stay, bool masked, int first) {
    Parts<kParts> ip[2], op[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      ip[k] = F::template get<kParts, typename F::Rows>(s.in, k);
      op[k] = F::template get<kParts, typename F::Rows>(s.out, k);
    }
#pragma unroll
    for (int j = 0; j < F::own; ++j)
      if (F::tile(j) < F::DT) {
        f32x4_t n, more = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) n[i] = times(stay, state[j][i]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          Parts<NP> qt = F::cols_of(s.q, F::tile(j), k), kt = F::cols_of(s.k, F::tile(j), k);
          if (masked) keep(qt, 32 * k + 8 * q4, 0, first), keep(kt, 32 * k + 8 * q4, 0, first);
          n = mma(qt, ip[k], n);
          more = mma(kt, op[k], more);
        }
        state[j] = n + more;
      }
    F::put_state(s.state, state);
  }

  __device__ __forceinline__ void chunk(int c, int next, Chunk& x) {
    f32x4_t dy = dy_of(c, x);
    F::template put<NP, typename F::Rows>(s.dy, row(), dy);
    __syncthreads();  // the state's parts and dy are there
    const Gates gates = F::load_gates(next);
    F::put_rows(s.k, x.k);
    F::put_rows(s.q, x.q);
    f32x4_t kd = {0.f, 0.f, 0.f, 0.f}, more = kd;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const auto sp = F::template get<kParts, typename F::State>(s.state, k);
      (k & 1 ? more : kd) = mma(F::rows_of(x.k, k), sp, k & 1 ? more : kd);
    }
    kd += more;
    fetch_rows(next, x);
    // All rows at once, and where something is not finite once more, each sequence by itself, so that nothing crosses a
    // start.  `first`: the rows that the state before the chunk reaches are those of the first sequence.
    f32x4_t z;
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
      float test = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) test = fmaf(z[i], 0.f, test);
      give(c, x, z, dy);
      if (__any(test != 0.f)) s.bad[turn & 1] = 1;  // NaN
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
    F::template load_matrix<true>(a.w.solve_t, next, x.solve);
    F::template load_matrix<true>(a.w.read_t, next, x.read);
    move(x.g.stay, masked, first);
    // stores come after the loads of the next chunk (see delta_fwd.h)
    store(c, x.g.beta, z);
    keep_state(c - 1);
    x.g = gates;
  }
  // The gradient of the state after chunk c.
  __device__ __forceinline__ void keep_state(int c) const {
    F::store_state(c >= 0 ? a.w.dstate + chunk_index(a, F::bh, c) * a.dk * a.dvp : nullptr, a.dvp, a.dvp, state);
  }
};

template <typename T, int DK>
__global__ __launch_bounds__(kTeam, 2) void delta_bwd_kernel(DeltaArgs a, int blocks) {
  typedef Backward<T, DK> F;
  __shared__ __attribute__((aligned(16))) typename F::Lds s;
  int bh, cb;
  if (!head_of(a.b * a.hv, blocks, bh, cb)) return;
  F f(a, s, bh, cb);
  const int64_t size = (int64_t)a.dk * a.dv;
  f.load_state(a.dh_last ? a.dh_last + bh * size : nullptr, f.state);
  if (threadIdx.x == 0) s.bad[0] = s.bad[1] = 0;
  f.put_state(s.state, f.state);
  if (a.chunks > 0) {
    typename F::Chunk x;
    f.fetch(a.chunks - 1, x);
    f.keep_state(a.chunks - 1);
    for (int c = a.chunks - 1; c >= 0; --c) f.chunk(c, max(c - 1, 0), x);
  }
  f.store_state(a.dh0 + bh * size, a.dv, a.dv, f.state);
}

}  // namespace

template <typename T>
hipError_t delta_bwd_of(const DeltaArgs& a, hipStream_t s) {
  return for_dk(a.dk, [&](auto dk) {
    const int blocks = a.dvp / 16;
    hipLaunchKernelGGL((delta_bwd_kernel<T, decltype(dk)::value>), dim3((a.b * a.hv + 7) / 8 * 8 * blocks), dim3(kTeam), 0, s, a,
                       blocks);
    return hipGetLastError();
  });
}

}  // namespace convdelta
