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
    f32x4_t enter, leave, beta;
    float stay;
    T v[4];
  };

  Lds& s;
  f32x4_t state[F::own];
  int turn = 0;

  __device__ __forceinline__ Forward(const DeltaArgs& a_, Lds& s_, int bh_, int cb) : F(a_, bh_, cb), s(s_) {}

  __device__ __forceinline__ void fetch_gates(int c, Chunk& x) const {
    x.enter = F::load_gate(0, c);
    x.leave = F::load_gate(1, c);
    x.beta = F::load_gate(2, c);
    x.stay = a.w.rows[chunk_index(a, F::bh, c) * 4 * kChunk + kChunk - 1];
  }
  __device__ __forceinline__ void fetch(int c, Chunk& x) const {
    F::load_rows(a.k, c, x.k);
    F::load_rows(a.q, c, x.q);
    F::template load_matrix<false>(a.w.solve, c, x.solve);
    F::template load_matrix<false>(a.w.read, c, x.read);
    fetch_gates(c, x);
    F::load_col(a.v, c, x.v);
  }

  // One chunk, all of its rows, or (`alone`) row `only` of it.  False where u is not finite: the state is then as it
  // was.  x holds chunk `next` afterwards.
  __device__ __forceinline__ bool chunk(int c, int next, Chunk& x, bool alone, int only) {
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    if (alone) {
      // a row by itself: its own decay takes the place of the sums', and only its products count
      x.enter = F::load_gate(3, c);
      x.stay = a.w.rows[(chunk_index(a, F::bh, c) * 4 + 3) * kChunk + only];
#pragma unroll
      for (int i = 0; i < 4; ++i) x.leave[i] = row() + i == only ? 1.f : 0.f;
    }
    __syncthreads();  // the state's parts are there
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
      xs[i] = to_f32(x.v[i]) - times(x.enter[i], ks[i]);
      u[i] = alone && row() + i != only ? 0.f : x.beta[i] * xs[i];
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
      for (int i = 0; i < 4; ++i) u[i] = x.beta[i] * xs[i];
    }
    F::template load_matrix<false>(a.w.solve, next, x.solve);
    f32x4_t lu;
    float test = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lu[i] = times(x.leave[i], u[i]);
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
        for (int i = 0; i < 4; ++i) n[i] = times(x.stay, state[j][i]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          Parts<NP> kt = F::cols_of(s.k, F::tile(j), k);
          if (alone) keep(kt, 32 * k + 8 * q4, only, only + 1);
          (k ? more : n) = mma(kt, up[k], k ? more : n);
        }
        state[j] = n + more;
      }
    F::put_state(s.state, state);
    f32x4_t o, more = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = times(x.enter[i], qs[i]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (F::template has<false>(k)) {
        if (alone) keep(x.read[k], 32 * k + 8 * q4, only, only + 1);
        const auto op = F::template get<YP, typename F::Rows>(s.out, k);
        (k ? more : o) = mma_first<YP>(x.read[k], op, k ? more : o);
      }
    const int64_t ld = (int64_t)a.hv * a.dv;
    T* y = (T*)a.y + ((int64_t)F::b * a.t + c * kChunk) * ld + (int64_t)F::h * a.dv;
    const uint32_t to = (uint32_t)(row() * (uint32_t)ld + col) * (uint32_t)sizeof(T);
    const int n = a.t - c * kChunk;
    if (F::live)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row() + i < n && (!alone || row() + i == only)) store_at(y + i * ld, to, from_f32<T>(a.scale * (o[i] + more[i])));
    F::template load_matrix<false>(a.w.read, next, x.read);
    fetch_gates(next, x);
    return true;
  }

  // The chunks [c, end), x holding chunk c.  One in which something is not finite goes row by row, so that it reaches
  // only what comes after it.
  template <typename Before>
  __device__ __forceinline__ void run(int c, int end, Chunk& x, const Before& before) {
    bool alone = false;
    int only = 0;
#pragma clang loop unroll(disable)
    while (c < end) {
      const int n = min(kChunk, a.t - c * kChunk);
      const bool last = !alone || only + 1 >= n;
      if (!alone) before(c);
      if (!chunk(c, last ? min(c + 1, end - 1) : c, x, alone, only)) {
        alone = true;
        only = 0;
        fetch(c, x);
        continue;
      }
      if (last) {
        ++c;
        alone = false;
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
  typename F::Chunk x;
  if (a.chunks > 0) f.fetch(0, x);
  f.run(0, a.chunks, x, [&](int c) {
    if (a.states) f.store_state(a.states + (((int64_t)f.b * a.chunks + c) * a.hv + f.h) * size, a.dv, f.live, f.state);
  });
  f.store_state(a.h_last + bh * size, a.dv, f.live, f.state);
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
