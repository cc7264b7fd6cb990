// delta_fwd.h -- gated delta rule forward: a workgroup carries 16 columns of one
// head's state through the chunks.  Included by one source for each type.
//
// A chunk takes three steps between barriers: (1) k S and q S, r; (2) x = r + H (beta r),
// u; (3) the state, y.  Each wave has its own rows (1, 2, y) or rows of the state (3), and
// fetches the next chunk's operands, each of which no other wave needs, as soon as this
// chunk's are used.
#include "delta_team.h"

namespace convdelta {

namespace {

template <typename T, int DK>
struct FwdLds {
  typedef Team<T, DK> F;
  __bf16 k[F::NP * RowsAt<DK>::part];
  __bf16 state[kParts * F::State::part];
  __bf16 br[kParts * F::Rows::part], u[kParts * F::Rows::part], out[F::YP * F::Rows::part];
  int bad[2];
};

template <typename T, int DK>
struct Forward : Team<T, DK> {
  typedef Team<T, DK> F;
  typedef FwdLds<T, DK> Lds;
  using F::a;
  using F::q4;
  using F::m;
  using F::wave;
  using F::col;
  using F::row;
  static constexpr int NP = F::NP, KS = F::KS, YP = F::YP;

  // what a chunk needs
  struct Chunk {
    Raw8<T> k[KS], q[KS];
    Parts<kParts> solve[2];
    Parts<YP> read[2];
    Gates g;
    T v[4];
  };

  Lds& s;
  f32x4_t state[F::own];
  int turn = 0;

  __device__ __forceinline__ Forward(const DeltaArgs& a_, Lds& s_, int bh_, int cb) : F(a_, bh_, cb), s(s_) {}

  __device__ __forceinline__ void fetch(int c, Chunk& x) const {
    F::load_rows(a.k, c, x.k);
    F::load_rows(a.q, c, x.q);
    F::template load_matrix<false>(a.w.solve, c, x.solve);
    F::template load_matrix<false>(a.w.read, c, x.read);
    x.g = F::load_gates(c);
    F::load_col(a.v, c, x.v);
  }

  // One chunk, all of its rows, or (`alone`) row `only` of it.  False where u is not finite: the state is then as it
  // was.  x holds chunk `next` afterwards.
  __device__ __forceinline__ bool chunk(int c, int next, Chunk& x, bool alone, int only) {
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    if (alone) {
      // a row by itself: its own decay takes the place of the sums', and only its products count
      x.g.enter = F::load_gate(3, c);
      x.g.stay = a.w.rows[(chunk_index(a, F::bh, c) * 4 + 3) * kChunk + only];
#pragma unroll
      for (int i = 0; i < 4; ++i) x.g.leave[i] = row() + i == only ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (unsigned n = 0; n < sizeof(T) / 2; ++n)
          if (16 * wave + m != only) x.k[k].w[n] = convfwd::u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int k = 0; k < 2; ++k) keep(x.read[k], 32 * k + 8 * q4, only, only + 1);
      wait_for_memory();
    }
    __syncthreads();  // the state's parts are there
    const Gates gates = F::load_gates(next);
    F::put_rows(s.k, x.k);
    f32x4_t ks = zero, qs = zero;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const auto sp = F::template get<kParts, typename F::State>(s.state, k);
      ks = mma(F::rows_of(x.k, k), sp, ks);
      qs = mma_first<YP>(F::rows_of(x.q, k), sp, qs);
    }
    f32x4_t xs, u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xs[i] = to_f32(x.v[i]) - times(x.g.enter[i], ks[i]);
      u[i] = alone && row() + i != only ? 0.f : x.g.beta[i] * xs[i];
    }
    F::load_rows(a.k, next, x.k);
    F::load_rows(a.q, next, x.q);
    F::load_col(a.v, next, x.v);
    F::template put<kParts, typename F::Rows>(s.br, row(), u);
    __syncthreads();
    if (!alone) {
      f32x4_t more = zero;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (F::template has<false>(k)) {
          const auto bp = F::template get<kParts, typename F::Rows>(s.br, k);
          (k ? more : xs) = mma(x.solve[k], bp, k ? more : xs);
        }
      xs += more;
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = x.g.beta[i] * xs[i];
    }
    F::template load_matrix<false>(a.w.solve, next, x.solve);
    f32x4_t lu;
    float test = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lu[i] = times(x.g.leave[i], u[i]);
      test = fmaf(u[i], 0.f, test);
    }
    F::template put<YP, typename F::Rows>(s.out, row(), u);
    F::template put<kParts, typename F::Rows>(s.u, row(), lu);
    if (__any(test != 0.f)) s.bad[turn & 1] = 1;  // NaN
    __syncthreads();
    const bool bad = s.bad[turn & 1];
    // the other flag: read before the last barrier, set after the next one but one
    if (threadIdx.x == 0) s.bad[~turn & 1] = 0;
    ++turn;
    if (!alone && bad) return false;
    // the state moves on
    Parts<kParts> up[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) up[k] = F::template get<kParts, typename F::Rows>(s.u, k);
#pragma unroll
    for (int j = 0; j < F::own; ++j)
      if (F::tile(j) < F::DT) {
        f32x4_t n, more = zero;
#pragma unroll
        for (int i = 0; i < 4; ++i) n[i] = times(x.g.stay, state[j][i]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const auto kt = F::cols_of(s.k, F::tile(j), k);
          (k ? more : n) = mma(kt, up[k], k ? more : n);
        }
        state[j] = n + more;
      }
    F::put_state(s.state, state);
    f32x4_t o, more = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = times(x.g.enter[i], qs[i]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (F::template has<false>(k)) {
        if (alone) keep(x.read[k], 32 * k + 8 * q4, only, only + 1);
        const auto op = F::template get<YP, typename F::Rows>(s.out, k);
        (k ? more : o) = mma_first<YP>(x.read[k], op, k ? more : o);
      }
    // Stores come after the loads of the next chunk: waits for memory are counted in the order of issue, and a load
    // issued after a store would be waited for together with it.
    F::template load_matrix<false>(a.w.read, next, x.read);
    x.g = gates;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = a.scale * (o[i] + more[i]);
    F::store_col(a.y, c, o, alone ? only : 0, alone ? only + 1 : kChunk);
    return true;
  }

  // The state before chunk c, kept for the backward pass.
  __device__ __forceinline__ void keep_state(int c) const {
    float* to = a.states && c < a.chunks ? a.states + (((int64_t)F::b * a.chunks + c) * a.hv + F::h) * a.dk * a.dv : nullptr;
    F::store_state(to, a.dv, a.dv, state);
  }

  // All chunks, x holding the first.  One in which something is not finite goes row by row, so that it reaches only
  // what comes after it.
  __device__ __forceinline__ void run(Chunk& x) {
    bool alone = false;
    int c = 0, only = 0;
    keep_state(0);
#pragma clang loop unroll(disable)
    while (c < a.chunks) {
      const bool last = !alone || only + 1 >= min(kChunk, a.t - c * kChunk);
      if (!chunk(c, last ? min(c + 1, a.chunks - 1) : c, x, alone, only)) {
        alone = true;
        only = 0;
        fetch(c, x);
        wait_for_memory();
        continue;
      }
      if (last) {
        ++c;
        alone = false;
        keep_state(c);
      } else {
        ++only;
      }
    }
  }
};

template <typename T, int DK>
__global__ __launch_bounds__(kTeam, 2) void delta_fwd_kernel(DeltaArgs a, int blocks) {
  typedef Forward<T, DK> F;
  __shared__ __attribute__((aligned(16))) typename F::Lds s;
  int bh, cb;
  if (!head_of(a.b * a.hv, blocks, bh, cb)) return;
  F f(a, s, bh, cb);
  const int64_t size = (int64_t)a.dk * a.dv;
  f.load_state(a.h0 ? a.h0 + bh * size : nullptr, f.state);
  if (threadIdx.x == 0) s.bad[0] = s.bad[1] = 0;
  f.put_state(s.state, f.state);
  if (a.chunks > 0) {
    typename F::Chunk x;
    f.fetch(0, x);
    f.run(x);
  }
  f.store_state(a.h_last + bh * size, a.dv, a.dv, f.state);
}

}  // namespace

template <typename T>
hipError_t delta_fwd_of(const DeltaArgs& a, hipStream_t s) {
  return for_dk(a.dk, [&](auto dk) {
    const int blocks = (a.dv + 15) / 16;
    hipLaunchKernelGGL((delta_fwd_kernel<T, decltype(dk)::value>), dim3((a.b * a.hv + 7) / 8 * 8 * blocks), dim3(kTeam), 0, s, a,
                       blocks);
    return hipGetLastError();
  });
}

}  // namespace convdelta
