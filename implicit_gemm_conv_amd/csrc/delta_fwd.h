// delta_fwd.h -- gated delta rule forward: a workgroup carries 16 or 32 columns of one
// head's state through the chunks.  Included by one source for each type.
//
// A chunk takes three steps between barriers: (1) k S and r; (2) x = r + H (beta r), u;
// (3) the state.  The waves of the first role go the way from state to state (k S, r, x, u);
// those of the second compute q S in step (2) and finish y in step (1) of the next chunk, while
// the first role is at work; the state's rows are all waves'.  Each wave fetches what it needs
// of the next chunk, which no other wave needs, as soon as this chunk's is used.
//
// Why columns: the columns of a state go their own ways through the sequence, so splitting them
// needs no exchange, and it is the only axis besides the heads that a single sequence offers; what it
// costs is that q, k and the chunks' matrices are read by every workgroup of a head, which sit on
// one die and share its L2.  States in fp32 (accumulators in registers, three bf16 parts in LDS for
// the products), matrices in three parts, on y's way too: q S and R u may cancel, and two parts there leave 2^-17 of
// their terms in a 16-bit y (with them the sequence below took 545 us).
//
// Bound by the chain of a chunk's steps: LDS, two to four matrix instructions one after the other,
// LDS, a barrier, three times over, about 4900 clocks a chunk (on the CUs in use matrix units busy 16%, vector units 26%).
// One sequence of 16387 rows, 16 heads of 128 x 128, bf16: 595 us, 2.3 us a chunk (prefill, 128
// workgroups on 256 CUs); 4 sequences of 4096, states kept: 316 us, 2.1 TB/s of HBM traffic.
#include "delta_team.h"

namespace convdelta {

namespace {

template <typename T, int DK, int NC>
struct FwdLds {
  typedef Team<T, DK, NC> F;
  __bf16 k[F::NP * RowsAt<DK>::part];
  __bf16 state[NC][kParts * F::State::part];
  __bf16 br[NC][kParts * F::Rows::part], u[NC][kParts * F::Rows::part], out[2][NC][kParts * F::Rows::part];
  int bad[2];
};

template <typename T, int DK, int NC, bool FIRST, bool TRAIN>
struct Forward : Team<T, DK, NC> {
  typedef Team<T, DK, NC> F;
  typedef FwdLds<T, DK, NC> Lds;
  using F::a;
  using F::q4;
  using F::m;
  using F::wave;
  using F::row;
  static constexpr int NP = F::NP, KS = F::KS;
  typedef typename F::Rows Rows;

  // what a chunk needs
  struct Chunk {
    Raw8<T> rows[KS];      // of k, or of q
    Parts<kParts> mat[2];  // of H; of the decayed q k^T of the chunk whose y is next
    f32x4_t enter, leave, beta;
    float stay;
    T v[NC][4];
  };

  Lds& s;
  f32x4_t state[NC], read[NC];
  int turn = 0, was = 0, was_first = 0, was_end = 0;  // the chunk whose y is to be finished

  __device__ __forceinline__ Forward(const DeltaArgs& a_, Lds& s_, int bh_, int cb) : F(a_, bh_, cb), s(s_) {}

  __device__ __forceinline__ void fetch_rows(int c, Chunk& x) const {
    F::load_rows(FIRST ? a.k : a.q, c, x.rows);
    if (FIRST) F::load_col(a.v, c, x.v);
  }
  __device__ __forceinline__ void fetch_matrix(int c, Chunk& x) const {
    F::template load_matrix<false>(FIRST ? a.w.solve : a.w.read, c, x.mat);
  }

  // What is loaded next takes its registers over: a load that moves up, past the last use of what they hold, takes
  // others, and its result has to be waited for and moved at the turn's end.  So has one whose use moves down.
  static __device__ __forceinline__ void used() { __builtin_amdgcn_sched_barrier(0); }
  static __device__ __forceinline__ void used(f32x4_t& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float e = v[i];
      asm volatile("" : "+v"(e));
      v[i] = e;
    }
  }

  // y of the chunk before, of its rows [first, end): what q S was is in `read`, u in LDS.
  __device__ __forceinline__ void finish(int c, const Chunk& x, int first, int end) const {
    f32x4_t y[NC], more[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) y[n] = read[n], more[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (F::template has<false>(k)) {
        Parts<kParts> mat = x.mat[k];
        if (end - first < kChunk) keep(mat, 32 * k + 8 * q4, first, end);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const auto op = F::template get<kParts, Rows>(s.out[~turn & 1][n], k);
          (k ? more : y)[n] = mma(mat, op, (k ? more : y)[n]);
        }
      }
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[n][i] = a.scale * (y[n][i] + more[n][i]);
    F::template store_col<T>(a.y, c, y, first, end);
  }

  // One chunk, all of its rows, or (`alone`) row `only` of it.  False where u is not finite: the state is then as it
  // was.  x holds chunk `next` afterwards.
  __device__ __forceinline__ bool chunk(int c, int next, Chunk& x, bool alone, int only) {
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    if (alone) {
      // a row by itself: its own decay takes the place of the sums', and only its products count
      if (FIRST) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x.leave[i] = row() + i == only ? 1.f : 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (unsigned n = 0; n < sizeof(T) / 2; ++n)
            if (16 * wave + m != only) x.rows[k].w[n] = convfwd::u32x4_t{0u, 0u, 0u, 0u};
      }
      wait_for_memory();
    }
    __syncthreads();  // the state's parts are there
    if (FIRST) F::put_rows(s.k, x.rows);
    f32x4_t xs[NC], more[NC];  // k S, or q S; then r, x
    float stay = x.stay;
    const auto times_state = [&] {
#pragma unroll
      for (int n = 0; n < NC; ++n) xs[n] = more[n] = zero;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const Parts<NP> rows = F::rows_of(x.rows, k);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          f32x4_t& to = (k & 1 ? more : xs)[n];
          const auto sp = F::template get<kParts, typename F::State>(s.state[n], k);
          to = mma(rows, sp, to);
        }
      }
      f32x4_t enter = x.enter;
      if (alone) {
        enter = F::load_gate(3, c);
        stay = a.w.rows[(chunk_index(a, F::bh, c) * 4 + 3) * kChunk + only];
        wait_for_memory();
      }
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // alone: a state that is not finite, behind a start (with all rows such a chunk comes to nothing)
          xs[n][i] = alone && enter[i] == 0.f ? 0.f : enter[i] * (xs[n][i] + more[n][i]);
          if (alone && stay == 0.f) state[n][i] = 0.f;
        }
    };
    f32x4_t u[NC], lu;
    if constexpr (FIRST) {
      times_state();
#pragma unroll
      for (int n = 0; n < NC; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xs[n][i] = to_f32(x.v[n][i]) - xs[n][i];
          u[n][i] = alone && row() + i != only ? 0.f : x.beta[i] * xs[n][i];
        }
        F::template put<kParts, Rows>(s.br[n], row(), u[n]);
      }
      used();
      x.enter = F::load_gate(0, next);
      fetch_rows(next, x);
    } else {
      finish(was, x, was_first, was_end);
      used();
      fetch_matrix(c, x);
    }
    __syncthreads();
    const float stay_next = F::load_stay(next);
    if (FIRST) {
      if (!alone) {
        // sums of their own, added to r (and to the state) once: a sum that starts from them is rounded to their size at
        // every product
        f32x4_t hx[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) hx[n] = more[n] = zero;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (F::template has<false>(k))
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              const auto bp = F::template get<kParts, Rows>(s.br[n], k);
              (k ? more : hx)[n] = mma(x.mat[k], bp, (k ? more : hx)[n]);
            }
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          xs[n] += hx[n] + more[n];
#pragma unroll
          for (int i = 0; i < 4; ++i) u[n][i] = x.beta[i] * xs[n][i];
        }
      }
      float test = 0.f;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lu[i] = x.leave[i] * u[n][i];
          test = fmaf(u[n][i], 0.f, test);
        }
        F::template put<kParts, Rows>(s.u[n], row(), lu);
        F::template put<kParts, Rows>(s.out[turn & 1][n], row(), u[n]);
      }
      if (__any(test != 0.f)) s.bad[turn & 1] = 1;  // NaN
    } else {
      times_state();
#pragma unroll
      for (int n = 0; n < NC; ++n) used(read[n] = xs[n]);
      used();
      x.enter = F::load_gate(0, next);
      fetch_rows(next, x);
    }
    // what the state's step has of k, which is there already, and all that is left to load
    Parts<NP> kt[2];
    if (F::has_tile())
#pragma unroll
      for (int k = 0; k < 2; ++k) kt[k] = F::cols_of(s.k, F::tile, k);
    used();
    if (FIRST) {
      x.leave = F::load_gate(1, next);
      x.beta = F::load_gate(2, next);
      fetch_matrix(next, x);
    }
    __syncthreads();
    const bool bad = s.bad[turn & 1];
    // the other flag: read before the last barrier, set after the next one but one
    if (threadIdx.x == 0) s.bad[~turn & 1] = 0;
    ++turn;
    was_end = was_first;
    if (!alone && bad) return false;
    was = c;
    was_first = alone ? only : 0;
    was_end = alone ? only + 1 : kChunk;
    // the state moves on
    if (F::has_tile()) {
      f32x4_t ku[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) ku[n] = more[n] = zero;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const auto up = F::template get<kParts, Rows>(s.u[n], k);
          (k ? more : ku)[n] = mma(kt[k], up, (k ? more : ku)[n]);
        }
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) state[n][i] = fmaf(stay, state[n][i], ku[n][i] + more[n][i]);
      F::put_state(s.state, state);
    }
    // Stores come after the loads of the next chunk: waits for memory are counted in the order of issue, and a load
    // issued after a store would be waited for together with it.
    if (FIRST && TRAIN) F::template store_col<float>(a.x, c, xs, was_first, was_end);
    x.stay = stay_next;
    return true;
  }

  // The state before chunk c, kept for the backward pass.
  __device__ __forceinline__ void keep_state(int c) const {
    if (!TRAIN) return;
    float* to = c < a.chunks ? a.states + (((int64_t)F::b * a.chunks + c) * a.hv + F::h) * a.dk * a.dv : nullptr;
    F::store_state(to, a.dv, a.dv, state);
  }
  __device__ __forceinline__ void fetch(int c, Chunk& x) const {
    fetch_rows(c, x);
    if (FIRST) {
      fetch_matrix(c, x);
      x.leave = F::load_gate(1, c);
      x.beta = F::load_gate(2, c);
    }
    x.enter = F::load_gate(0, c);
    x.stay = F::load_stay(c);
  }

  // All chunks.  One in which something is not finite goes row by row, so that it reaches only what comes after it.
  // (Both roles take the same turns: they wait for each other at every barrier.)
  __device__ __forceinline__ void run() {
    const int64_t size = (int64_t)a.dk * a.dv;
    F::load_state(a.h0 ? a.h0 + F::bh * size : nullptr, state);
    F::put_state(s.state, state);
    if (a.chunks > 0) {
      Chunk x;
      fetch(0, x);
      if (!FIRST) fetch_matrix(0, x);
#pragma unroll
      for (int n = 0; n < NC; ++n) read[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
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
      if constexpr (!FIRST) finish(was, x, was_first, was_end);
    }
    F::store_state(a.h_last + F::bh * size, a.dv, a.dv, state);
  }
};

template <typename T, int DK, int NC, bool TRAIN>
__global__ __launch_bounds__(kTeam, 2) void delta_fwd_kernel(DeltaArgs a, int blocks) {
  __shared__ __attribute__((aligned(16))) FwdLds<T, DK, NC> s;
  int bh, cb;
  if (!head_of(a.b * a.hv, blocks, bh, cb)) return;
  if (threadIdx.x < 2) s.bad[threadIdx.x] = 0;
  if (wave_id() < 4)
    Forward<T, DK, NC, true, TRAIN>(a, s, bh, cb).run();
  else
    Forward<T, DK, NC, false, TRAIN>(a, s, bh, cb).run();
}

}  // namespace

template <typename T>
hipError_t delta_fwd_of(const DeltaArgs& a, hipStream_t s) {
  return for_dk(a.dk, [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    return for_columns(a, [&](auto nc) {
      constexpr int NC = decltype(nc)::value;
      const int blocks = (a.dv + 16 * NC - 1) / (16 * NC);
      hipLaunchKernelGGL((a.states ? delta_fwd_kernel<T, DK, NC, true> : delta_fwd_kernel<T, DK, NC, false>),
                         dim3((a.b * a.hv + 7) / 8 * 8 * blocks), dim3(kTeam), 0, s, a, blocks);
      return hipGetLastError();
    });
  });
}

}  // namespace convdelta
