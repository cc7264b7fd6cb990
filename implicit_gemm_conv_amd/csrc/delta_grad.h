// delta_grad.h -- gated delta rule, the gradients that add over all columns of v: one
// workgroup of eight waves a chunk and key head, all chunks at once.  With S the state
// before the chunk, dS the gradient of the one after it, x what the forward pass kept,
// u = beta x, dx = beta z,
//
//   dP = scale * D * (dy u^T) (j <= i),  dL = -D * (dx u^T) (j < i)
//   dq = scale * enter * (dy S^T) + dP k
//   dk = -enter * (dx S^T) + leave * (u dS^T) + dL k + dL^T k + dP^T q
//   dbeta = z . x
//
// The gradient of a row's log decay is the sum of all terms that its decay is a factor of: with
//   e_i = scale * enter_i (q_i S) . dy_i - enter_i (k_i S) . dx_i,  f_j = leave_j k_j . (dS u_j)
//   M_ij = dP_ij (q_i . k_j) + dL_ij (k_i . k_j)  (j < i)
// dlog_decay_i is the sum of e_l over l >= i, of f_j over j < i, of M_lj over l >= i > j, and stay * <S, dS>.  Every term is
// as much decayed as the gradient itself, so that its error is fp32's relative to it also where the decay is
// next to nothing.  (The same as a difference, <S, its gradient> less the rows' q . dq - dx . v, has the error of what is
// subtracted: with decays of e^-16 it is mostly rounding.)
//
// The columns are taken 32 at a time, through LDS (one slice there: with two, which fit up to Dk = 64, both
// passes took 954 us for 953 at Dk = 64); wave (w, half) owns rows 16 w .. + 15 and half of dq's and dk's
// columns.  All operands have three parts: with two in what ends in a 16-bit dk alone (2^-17 of its terms) both passes
// took 30 us less of 1221 at the size below.
//
// 4 sequences of 4096 rows, 16 heads of 128 x 128, bf16: 504 us, 1.4 TB/s of HBM traffic.  (Reading x instead of
// solving for it again took 830 to 534 us, loads of a slice ahead of its products 495 us, decays without branches
// 471 us, all of them with two parts in dk's operands; three added 30 us.)  Bound by vector work (busy
// 43%: parts of fp32 values for the matrix units; these 17%) in turns with LDS, in one workgroup of 226 registers
// a CU, whose start and end nothing covers.  Included by one source for each type.
#include "delta_team.h"

namespace convdelta {

namespace {

constexpr int kT = 512, kCols = 32, kSlice = kCols + 8, kLdM = kChunk + 8;

template <typename T, int DK>
struct GradLds {
  typedef Team<T, DK, 1> F;
  static constexpr int NP = F::NP;
  union {
    struct {
      __bf16 s[kParts * DK * kSlice], ds[kParts * DK * kSlice];          // 32 columns of both states, rows d
      __bf16 u[kParts * kChunk * kSlice], dx[kParts * kChunk * kSlice];  // rows of the chunk
    } slice;
    struct {
      __bf16 p[kParts * kChunk * kLdM], l[kParts * kChunk * kLdM];       // dP and dL
      __bf16 k[NP * RowsAt<DK>::part], q[NP * RowsAt<DK>::part];
    };
  };
  float gates[2 * kChunk], zx[kChunk];  // enter, leave; z.x
  float red[3][2][kChunk];              // both halves' shares of e, f and the sums of M
  float after[3][kChunk];               // sums of M's columns over the rows of the waves 1, 2 and 3
  double sums[kChunk], a[kT / 64];
  int seq[kChunk], wild;
};

template <typename T, int DK, bool WHOLE>
struct Grad {
  typedef Team<T, DK, 1> F;
  typedef GradLds<T, DK> Lds;
  static constexpr int NP = F::NP, DT = DK / 32;  // DT: 16-row tiles of a half of dq's columns
  static constexpr int each = DK * kCols / 4 / kT;                          // pieces of 4 floats of a slice a thread
  static_assert(each >= 1 || DK == 32, "slices");
  static constexpr int held = each ? each : 1;

  const DeltaArgs& a;
  Lds& s;
  int wave, half, lane, m, q4, b, c, own, tid;  // own: the lane's first row of accumulators

  __device__ __forceinline__ Grad(const DeltaArgs& a_, Lds& s_, int b_, int c_) : a(a_), s(s_), b(b_), c(c_) {
    const int w = wave_id();
    wave = w % 4;
    half = w / 4;
    renew();
  }
  // Where the lane stands, as something new: what the compiler makes of it (addresses, mostly) is made again
  // where it is needed next, and not held in registers, or spilled, from the kernel's start on.
  __device__ __forceinline__ void renew() {
    tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    lane = tid % 64;
    m = lane % 16;
    q4 = lane / 16;
    own = 16 * wave + 4 * q4;
  }

  // What a slice of 32 columns is made of: pieces of both states; 4 columns of a row of z and x; 8 of the lane's row of
  // dy, an operand.
  struct Slice {
    f32x4_t st[held], ds[held], z, x;
    Raw8<T> dy;
  };
  // N neighbouring elements of a row, zero past its end: as pieces of at most 16 bytes, where rows are whole ones (WHOLE)
  // or of fp32, whose pieces need no more than their own alignment (4x4096 rows, 16 heads of 128 x 128, bf16: 842 us for
  // the whole backward pass, 915 with dy element by element).
  template <typename E, int N>
  __device__ __forceinline__ void load(const Range& x, uint32_t row, int col, int width, void* to) const {
    constexpr int n = WHOLE || sizeof(E) == 4 ? (N * sizeof(E) > 16 ? 16 / sizeof(E) : N) : 1;
    struct alignas(n * sizeof(E)) Piece { E e[n]; };
#pragma unroll
    for (int k = 0; k < N / n; ++k) {
      const int at = col + k * n;
      Piece p = x.load<Piece>(at < width ? row + (uint32_t)at * (uint32_t)sizeof(E) : kNowhere);
      if constexpr (!WHOLE && n > 1)
#pragma unroll
        for (int e = 1; e < n; ++e)
          if (at + e >= width) p.e[e] = 0;
      __builtin_memcpy((E*)to + k * n, &p, sizeof(p));
    }
  }
  __device__ __forceinline__ void load_state(const Range& from, int v0, int ld, f32x4_t (&x)[held]) const {
#pragma unroll
    for (int k = 0; k < held; ++k) {
      const int i = tid + k * kT;
      load<float, 4>(from, (uint32_t)(i / 8 * ld) * 4u, v0 + i % 8 * 4, ld, &x[k]);  // rows past Dk are past the range
    }
  }
  template <int N>
  __device__ __forceinline__ void put_state(__bf16* to, const f32x4_t (&x)[held]) const {
#pragma unroll
    for (int k = 0; k < held; ++k) {
      const int i = tid + k * kT, d = i / (kCols / 4), v = i % (kCols / 4) * 4;
      if (d >= DK) continue;
      bf164_t o[N];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        __bf16 w[N];
        split_one<N>(x[k][e], w);
#pragma unroll
        for (int n = 0; n < N; ++n) o[n][e] = w[n];
      }
#pragma unroll
      for (int n = 0; n < N; ++n) *(bf164_t*)(to + (n * DK + d) * kSlice + v) = o[n];
    }
  }
  // 4 columns of a row of the chunk, as parts, into a slice
  template <int N>
  __device__ __forceinline__ void put_row(__bf16* to, const f32x4_t& x) const {
    bf164_t o[N];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      __bf16 w[N];
      split_one<N>(x[e], w);
#pragma unroll
      for (int n = 0; n < N; ++n) o[n][e] = w[n];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) *(bf164_t*)(to + (n * kChunk + tid / 8) * kSlice + tid % 8 * 4) = o[n];
  }
  // rows of a slice as an operand
  template <int N>
  __device__ __forceinline__ Parts<N> slice(const __bf16* x, int row, int part) const {
    return natural<N>(x + row * kSlice + 8 * q4, part * kSlice);
  }

  __device__ __forceinline__ float value(const __bf16* x, int r, int d) const {
    float v = 0.f;
#pragma unroll
    for (int n = NP - 1; n >= 0; --n) v += (float)x[n * RowsAt<DK>::part + r * RowsAt<DK>::stride + d];
    return v;
  }

  // out (own rows, own columns) += M x or M^T x, of M the first N parts; masked: over the rows [lo, hi), which are the
  // only ones added to
  template <bool UP, int N>
  __device__ __forceinline__ void add_range(const __bf16* mat, const __bf16* rows, f32x4_t (&out)[DT], bool masked, int lo, int hi) const {
    Parts<N> am[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      am[k] = UP ? transposed<N>(mat + (32 * k + 8 * q4 + m / 4) * kLdM + 16 * wave + 4 * (m % 4), kLdM, kChunk * kLdM)
                 : natural<N>(mat + (16 * wave + m) * kLdM + 32 * k + 8 * q4, kChunk * kLdM);
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      f32x4_t n = out[t];
      if (masked) n = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // a triangle: rows of this wave's tile hold nothing in the other half
        if (UP ? k < wave / 2 : k > wave / 2) continue;
        Parts<NP> bm = transposed<NP>(rows + (32 * k + 8 * q4 + m / 4) * RowsAt<DK>::stride + 16 * (half * DT + t) + 4 * (m % 4),
                                      RowsAt<DK>::stride, RowsAt<DK>::part);
        if (masked) keep(bm, 32 * k + 8 * q4, lo, hi);
        n = mma(am[k], bm, n);
      }
      if (masked) {
#pragma unroll
        for (int r = 0; r < 4; ++r) out[t][r] += own + r >= lo && own + r < hi ? n[r] : 0.f;
      } else {
        out[t] = n;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // with something in k or q that is not finite (wild), each sequence by itself
  template <bool UP, int N>
  __device__ __forceinline__ void add(const __bf16* mat, const __bf16* rows, f32x4_t (&out)[DT], bool wild) const {
    int hi = kChunk;
#pragma clang loop unroll(disable)
    do {
      int lo = 0;
      if (wild)
        for (lo = hi - 1; lo > 0 && s.seq[lo] == s.seq[lo - 1];) --lo;
      add_range<UP, N>(mat, rows, out, wild, lo, hi);
      hi = lo;
    } while (hi > 0);
  }

  // acc = factor * D * acc below (and, EDGE, on) the diagonal, zero elsewhere.  A half has the columns' tiles half, half + 2.
  template <bool EDGE>
  __device__ __forceinline__ void decayed(f32x4_t (&acc)[2], const f32x4_t (&decay)[2], float factor) const {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = 16 * (half + 2 * n) + m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool in = !(decay[n][r] < 0.f) && (EDGE ? j <= own + r : j < own + r);  // a NaN decay is wanted
        acc[n][r] = in ? factor * decay[n][r] * acc[n][r] : 0.f;
      }
    }
  }
  // ... as parts into LDS
  __device__ __forceinline__ void put_matrix(__bf16* to, const f32x4_t (&acc)[2]) const {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        __bf16 w[kParts];
        split_one<kParts>(acc[n][r], w);
#pragma unroll
        for (int p = 0; p < kParts; ++p) to[(p * kChunk + own + r) * kLdM + 16 * (half + 2 * n) + m] = w[p];
      }
  }
  // D of those tiles, -1 where the rows are not of one sequence
  __device__ __forceinline__ void get_decay(f32x4_t (&decay)[2]) const {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = 16 * (half + 2 * n) + m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = own + r;
        const float d = expf((float)(s.sums[i] - s.sums[j]));
        decay[n][r] = s.seq[i] == s.seq[j] ? d : -1.f;
      }
    }
  }

  __device__ __forceinline__ float over_lanes(float v) const {
    for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o);
    return v;
  }

  // M's columns of this wave's tiles, each element with those below it in the wave's 16 rows added
  __device__ __forceinline__ void columns_of_m(const f32x4_t (&dp)[2], const f32x4_t (&dl)[2], f32x4_t (&sum)[2]) const {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int tile = half + 2 * n;
      sum[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (tile > wave) continue;
      f32x4_t qk = sum[n], kk = sum[n];
#pragma unroll
      for (int e = 0; e < DK / 32; ++e) {
        const auto at = [&](const __bf16* x, int row) { return natural<NP>(x + row * RowsAt<DK>::stride + 32 * e + 8 * q4, RowsAt<DK>::part); };
        const auto kj = at(s.k, 16 * tile + m);
        qk = mma(at(s.q, 16 * wave + m), kj, qk);
        kk = mma(at(s.k, 16 * wave + m), kj, kk);
      }
      const int j = 16 * tile + m;
#pragma unroll
      for (int r = 3; r >= 0; --r)  // zeros of dP and dL stay zero, whatever a row of another sequence holds
        sum[n][r] = (j < own + r ? times(dp[n][r], qk[r]) + times(dl[n][r], kk[r]) : 0.f) + (r < 3 ? sum[n][r + 1] : 0.f);
      float below = 0.f;
#pragma unroll
      for (int o = 3; o >= 1; --o) {
        const float x = __shfl(sum[n][0], min(lane + 16 * o, 63));
        if (q4 + o < 4) below += x;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) sum[n][r] += below;
      if (wave > 0 && q4 == 0) s.after[wave - 1][j] = sum[n][0];
    }
  }

  // The gradients of one value head; its share of dq and dk.
  __device__ __forceinline__ void head(int hk, int h, f32x4_t (&dq)[DT], f32x4_t (&dk)[DT]) {
    const int64_t bh = (int64_t)b * a.hv + h, at = bh * a.chunks + c;
    const auto row = [&] { return 16 * wave + m; };  // the lane's row as an operand
    const int rows = min(kChunk, a.t - c * kChunk);
    const int64_t size = (int64_t)a.dk * a.dv, size_p = (int64_t)a.dk * a.dvp;
    const Range states(a.states_in + (((int64_t)b * a.chunks + c) * a.hv + h) * size, size * 4);
    const Range dstate(a.w.dstate + at * size_p, size_p * 4);
    const Range zs(a.w.z + at * kChunk * a.dvp, (int64_t)kChunk * a.dvp * 4);
    const Span kept = dense_rows(a, b, h, c, 4);
    const Range xs((const char*)a.x_in + kept.at, kept.bytes);
    const Range dys = rows_range<T>(a.dy, b, h, c * kChunk, a.t, a.dv);
    __syncthreads();  // what is read of the head before
    const float my_beta = load_at<float>(a.w.rows + (at * 4 + 2) * kChunk, (uint32_t)(tid / 8) * 4u);
    Slice x;
    const auto fetch = [&](int v0) {
      load_state(states, v0, a.dv, x.st);
      load_state(dstate, v0, a.dvp, x.ds);
      const int col = v0 + tid % 8 * 4;
      load<float, 4>(zs, (uint32_t)(tid / 8 * a.dvp) * 4u, col, a.dvp, &x.z);
      load<float, 4>(xs, (uint32_t)(tid / 8 * a.hv * a.dv) * 4u, col, a.dv, &x.x);
      load<T, 8>(dys, row() * row_bytes<T>(a.dy), v0 + 8 * q4, a.dv, x.dy.w);
    };
    Parts<NP> yp;
    float db = 0.f;
    double dot = 0;
    // what was fetched, into LDS, and dy into yp
    const auto put = [&] {
      auto& to = s.slice;
      put_state<kParts>(to.s, x.st);
      put_state<kParts>(to.ds, x.ds);
#pragma unroll
      for (int n = 0; n < held; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = fma((double)x.st[n][e], (double)x.ds[n][e], dot);
      f32x4_t u, dx;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = my_beta * x.x[e];
        dx[e] = my_beta * x.z[e];
        db = fmaf(x.x[e], x.z[e], db);
      }
      put_row<kParts>(to.u, u);
      put_row<kParts>(to.dx, dx);
      Raw8<T> dy = x.dy;
#pragma unroll
      for (unsigned n = 0; n < sizeof(T) / 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) dy.w[n][e] = row() < rows ? dy.w[n][e] : 0u;
      yp = dy.parts();
    };
    fetch(0);
    if (tid == 0) s.wild = 0;
    if (tid < 2 * kChunk) s.gates[tid] = a.w.rows[at * 4 * kChunk + tid];
    if (tid < kChunk) {
      s.sums[tid] = a.w.sums[at * kChunk + tid];
      s.seq[tid] = a.w.seq[at * kChunk + tid];
    }
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    f32x4_t dkr[DT], dkc[DT], dp[2] = {zero, zero}, dl[2] = {zero, zero};
#pragma unroll
    for (int t = 0; t < DT; ++t) dq[t] = dkr[t] = dkc[t] = zero;
    put();
    fetch(kCols);
    __syncthreads();
    Rows64<T, DK, kT> k, q;
#pragma clang loop unroll(disable)
    for (int v0 = 0; v0 < a.dvp; v0 += kCols) {
      renew();
      {
        auto& at = s.slice;
        const auto up = slice<kParts>(at.u, row(), kChunk);
        const auto xp = slice<kParts>(at.dx, row(), kChunk);
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          const int d = 16 * (half * DT + t) + m;
          const auto sp = slice<kParts>(at.s, d, DK);
          const auto dsp = slice<kParts>(at.ds, d, DK);
          dq[t] = mma(yp, sp, dq[t]);
          dkr[t] = mma(xp, sp, dkr[t]);
          dkc[t] = mma(up, dsp, dkc[t]);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
          if (half + 2 * n <= wave) {
            const auto uj = slice<kParts>(at.u, 16 * (half + 2 * n) + m, kChunk);
            dp[n] = mma(yp, uj, dp[n]);
            dl[n] = mma(xp, uj, dl[n]);
          }
      }
      if (v0 + kCols < a.dvp) {
        __syncthreads();  // what is read of the slice
        renew();
        put();
        __builtin_amdgcn_sched_barrier(0);  // the next slice takes this one's registers over
        fetch(v0 + 2 * kCols);
      } else {
        k.load(a.k, b, hk, c * kChunk, a.t, a.dkp);
        q.load(a.q, b, hk, c * kChunk, a.t, a.dkp);
      }
      __syncthreads();
    }
    renew();
    const f32x4_t enter = *(const f32x4_t*)(s.gates + own), leave = *(const f32x4_t*)(s.gates + kChunk + own);
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dq[t][r] = times(enter[r], a.scale * dq[t][r]);
        dkr[t][r] = times(enter[r], dkr[t][r]);
        dkc[t][r] = times(leave[r], dkc[t][r]);
      }
    for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o);
    if (lane == 0) s.a[4 * half + wave] = dot;
    for (int o = 1; o < 8; o <<= 1) db += __shfl_xor(db, o);
    if (tid % 8 == 0) s.zx[tid / 8] = db;
    if (!k.finite() || !q.finite()) s.wild = 1;
    {
      f32x4_t decay[2];
      get_decay(decay);
      renew();
      decayed<true>(dp, decay, a.scale);
      decayed<false>(dl, decay, -1.f);
    }
    put_matrix(s.p, dp);
    put_matrix(s.l, dl);
    k.put(s.k);
    q.put(s.q);
    __syncthreads();
    const bool wild = s.wild;
    renew();
    f32x4_t below[2];
    columns_of_m(dp, dl, below);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float e = 0.f, f = 0.f;
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const int d = 16 * (half * DT + t) + m;
        const float kd = value(s.k, own + r, d);
        e = fmaf(value(s.q, own + r, d), dq[t][r], e);
        e = fmaf(-kd, dkr[t][r], e);
        f = fmaf(kd, dkc[t][r], f);
      }
      e = over_lanes(e);
      f = over_lanes(f);
      // rows that the state does not reach, or that do not reach it, whatever they hold
      if (m == 0) s.red[0][half][own + r] = s.gates[own + r] == 0.f ? 0.f : e;
      if (m == 0) s.red[1][half][own + r] = s.gates[kChunk + own + r] == 0.f ? 0.f : f;
    }
#pragma unroll
    for (int t = 0; t < DT; ++t) dk[t] = dkc[t] - dkr[t];
    __syncthreads();
    renew();
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int w = 1; w < 4; ++w)
        if (half + 2 * n <= wave && wave < w) {
          const float x = s.after[w - 1][16 * (half + 2 * n) + m];
#pragma unroll
          for (int r = 0; r < 4; ++r) below[n][r] += x;
        }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float g = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (16 * (half + 2 * n) + m < own + r) g += below[n][r];
      g = over_lanes(g);
      if (m == 0) s.red[2][half][own + r] = g;
    }
    renew();
    add<false, kParts>(s.p, s.k, dq, wild);
    renew();
    add<false, kParts>(s.l, s.k, dk, wild);
    renew();
    add<true, kParts>(s.l, s.k, dk, wild);
    renew();
    add<true, kParts>(s.p, s.q, dk, wild);
    __syncthreads();
    if (tid < kChunk) {
      const int t = c * kChunk + lane;
      double e = (double)s.red[0][0][lane] + s.red[0][1][lane], f = (double)s.red[1][0][lane] + s.red[1][1][lane], all = 0;
      for (int o = 1; o < 64; o <<= 1) {
        const double x = __shfl_down(e, o), y = __shfl_up(f, o);
        if (lane + o < 64) e += x;
        if (lane >= o) f += y;
      }
      f = __shfl_up(f, 1);
      for (int w = 0; w < kT / 64; ++w) all += s.a[w];
      const float stay = s.gates[kChunk - 1];
      double g = e + ((double)s.red[2][0][lane] + s.red[2][1][lane]);
      if (lane > 0) g += f;
      if (stay != 0.f) g += stay * all;
      if (t < a.t) {
        const int64_t to = ((int64_t)b * a.t + t) * a.hv + h;
        a.dlog_decay[to] = (float)g;
        a.dbeta[to] = s.zx[lane];
      }
    }
  }
};

template <typename T, int DK, bool WHOLE>
__global__ __launch_bounds__(kT, 2) void delta_grad_kernel(DeltaArgs a) {
  typedef Grad<T, DK, WHOLE> F;
  __shared__ __attribute__((aligned(16))) typename F::Lds s;
  const int c = blockIdx.x % a.chunks, hk = blockIdx.x / a.chunks % a.hk, b = blockIdx.x / a.chunks / a.hk;
  F f(a, s, b, c);
  const int share = a.hv / a.hk;
  f32x4_t dq[F::DT], dk[F::DT], sq[F::DT], sk[F::DT];
  for (int n = 0; n < share; ++n) {
    f.head(hk, hk * share + n, dq, dk);
#pragma unroll
    for (int t = 0; t < F::DT; ++t) {
      sq[t] = n ? sq[t] + dq[t] : dq[t];
      sk[t] = n ? sk[t] + dk[t] : dk[t];
    }
  }
  const int64_t first = ((int64_t)b * a.t + c * kChunk) * a.hk + hk;
#pragma unroll
  for (int t = 0; t < F::DT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = f.own + r, d = 16 * (f.half * F::DT + t) + f.m;
      if (c * kChunk + row >= a.t || d >= a.dk) continue;
      const int64_t to = (first + (int64_t)row * a.hk) * a.dk + d;
      ((T*)a.dq)[to] = from_f32<T>(sq[t][r]);
      ((T*)a.dk_)[to] = from_f32<T>(sk[t][r]);
    }
}

}  // namespace

template <typename T>
hipError_t delta_grad_of(const DeltaArgs& a, hipStream_t s) {
  return for_dk(a.dk, [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    hipLaunchKernelGGL((a.whole ? delta_grad_kernel<T, DK, true> : delta_grad_kernel<T, DK, false>), dim3(a.b * a.hk * a.chunks),
                       dim3(kT), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace convdelta
