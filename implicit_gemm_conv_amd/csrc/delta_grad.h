// delta_grad.h -- gated delta rule, the gradients that add over all columns of v: one
// workgroup of eight waves a chunk and key head, all chunks at once.  With S the state
// before the chunk, dS the gradient of the one after it, x as in the forward pass (computed
// again from S), u = beta x, dx = beta z,
//
//   dP = scale * D * (dy u^T) (j <= i),  dL = -D * (dx u^T) (j < i)
//   dq = scale * enter * (dy S^T) + dP k
//   dk = -enter * (dx S^T) + leave * (u dS^T) + dL k + dL^T k + dP^T q
//   dbeta = z . x
//
// A row's decay scales what the row's q and v take part in, the one way and the other: with
// A the product <state before the chunk, its gradient>,
//
//   dlog_decay_i = A - sum over j < i of (q_j . dq_j - dx_j . v_j)
//
// and from zero at a start, where the decay acts on nothing.
//
// The columns are taken 32 at a time; wave (w, half) owns rows 16 w .. + 15 and half of
// the columns (of x) or of dq's and dk's.  What dlog_decay and dbeta are made of has fp32's
// precision (three parts); what ends in a 16-bit dk alone has two parts, 2^-17.
// Included by one source for each type.
#include "delta_team.h"

namespace convdelta {

namespace {

constexpr int kT = 512, kCols = 32, kSlice = kCols + 8, kLdM = kChunk + 8;

template <typename T, int DK>
struct GradLds {
  typedef Team<T, DK> F;
  static constexpr int NP = F::NP, GP = F::YP;
  __bf16 rows[NP * RowsAt<DK>::part];  // k, and at the end q
  union {
    struct {
      __bf16 s[kParts * DK * kSlice], ds[GP * DK * kSlice];          // 32 columns of both states, rows d
      __bf16 u[kParts * kChunk * kSlice], dx[GP * kChunk * kSlice];  // rows of the chunk
      __bf16 br[2 * kParts * F::Rows::part];                         // columns of beta r, 16 at a time
    };
    struct {
      __bf16 p[kParts * kChunk * kLdM], l[GP * kChunk * kLdM];       // dP and dL
    };
  };
  float gates[3 * kChunk], red[2][kChunk][3];  // enter, leave, beta; sums of both halves
  double sums[kChunk], a[kT / 64];
  int seq[kChunk], bad[2];
};

template <typename T, int DK>
struct Grad {
  typedef Team<T, DK> F;
  typedef GradLds<T, DK> Lds;
  static constexpr int NP = F::NP, GP = F::YP, KS = DK / 32, DT = DK / 32;  // DT: 16-row tiles of a half of dq's columns
  static constexpr int each = DK * kCols / 4 / kT;                          // pieces of 4 floats of a slice a thread
  static_assert(each >= 1 || DK == 32, "slices");
  static constexpr int held = each ? each : 1;

  const DeltaArgs& a;
  Lds& s;
  int wave, half, lane, m, q4, b, c, own, tid, turn = 0;  // own: the lane's first row of accumulators

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

  // 4 columns of row d of a (Dk, ld) state from column v0 on, whatever is there where it ends
  __device__ __forceinline__ void load_state(const float* from, int v0, int ld, f32x4_t (&x)[held]) const {
#pragma unroll
    for (int k = 0; k < held; ++k) {
      const int d = min(tid / (kCols / 4), a.dk - 1 - k * kT / (kCols / 4)), v = v0 + tid % (kCols / 4) * 4;
      const float* p = from + (int64_t)k * (kT / (kCols / 4)) * ld;
      if (k * kT / (kCols / 4) >= a.dk) continue;
      if (ld % 4 == 0) {
        x[k] = load_at<f32x4_t>(p, (uint32_t)(d * ld + min(v, ld - 4)) * 4u);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] = load_at<float>(p, (uint32_t)(d * ld + min(v + e, ld - 1)) * 4u);
      }
    }
  }
  // ... and zeros there
  __device__ __forceinline__ void within(f32x4_t (&x)[held], int v0, int width) const {
#pragma unroll
    for (int k = 0; k < held; ++k) {
      const int i = tid + k * kT, d = i / (kCols / 4), v = v0 + i % (kCols / 4) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[k][e] = d < a.dk && v + e < width ? x[k][e] : 0.f;
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
  // four rows of the lane's column, as parts, into rows of a slice
  template <int N>
  __device__ __forceinline__ void put_rows(__bf16* to, const f32x4_t& x) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __bf16 w[N];
      split_one<N>(x[i], w);
#pragma unroll
      for (int n = 0; n < N; ++n) to[(n * kChunk + own + i) * kSlice + 16 * half + m] = w[n];
    }
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
  __device__ __forceinline__ void add_range(const __bf16* mat, f32x4_t (&out)[DT], bool masked, int lo, int hi) const {
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
        Parts<NP> bm = transposed<NP>(s.rows + (32 * k + 8 * q4 + m / 4) * RowsAt<DK>::stride + 16 * (half * DT + t) + 4 * (m % 4),
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
  __device__ __forceinline__ void add(const __bf16* mat, f32x4_t (&out)[DT], bool wild) const {
    int hi = kChunk;
#pragma clang loop unroll(disable)
    do {
      int lo = 0;
      if (wild)
        for (lo = hi - 1; lo > 0 && s.seq[lo] == s.seq[lo - 1];) --lo;
      add_range<UP, N>(mat, out, wild, lo, hi);
      hi = lo;
    } while (hi > 0);
  }

  // M = factor * D * acc below (and, EDGE, on) the diagonal, as N parts into LDS.  A half has the columns' tiles half, half + 2.
  template <bool EDGE, int N>
  __device__ __forceinline__ void put_matrix(__bf16* to, const f32x4_t (&acc)[2], float factor) const {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = 16 * (half + 2 * n) + m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = own + r;
        const bool in = (EDGE ? j <= i : j < i) && s.seq[i] == s.seq[j];
        const float x = in ? factor * expf((float)(s.sums[i] - s.sums[j])) * acc[n][r] : 0.f;
        __bf16 w[N];
        split_one<N>(x, w);
#pragma unroll
        for (int p = 0; p < N; ++p) to[(p * kChunk + i) * kLdM + j] = w[p];
      }
    }
  }

  __device__ __forceinline__ float over_lanes(float v) const {
    for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o);
    return v;
  }

  // What a slice of 32 columns needs.
  struct Slice {
    f32x4_t s[held], ds[held], before[held], z;
    T v[4];
    Raw8<T> dy;
  };

  // The gradients of one value head; its share of dq and dk.
  __device__ __forceinline__ void head(int hk, int h, f32x4_t (&dq)[DT], f32x4_t (&dk)[DT]) {
    const int64_t bh = (int64_t)b * a.hv + h, at = bh * a.chunks + c;
    const auto row = [&] { return 16 * wave + m; };  // the lane's row as an operand
    Rows64<T, DK, kT> k, q;
    k.load(a.k, b, hk, c * kChunk, a.t, a.dkp);
    q.load(a.q, b, hk, c * kChunk, a.t, a.dkp);
    Parts<kParts> solve[2];
    {
      const char* p = a.w.solve + at * kMatrix + lane * 16;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int f = wave < 2 ? wave : 2 * wave - 2 + e;
#pragma unroll
        for (int n = 0; n < kParts; ++n) solve[e].p[n] = *(const bf168_t*)(p + (f * kParts + n) * kFrag);
      }
    }
    const float* states = a.states_in + (((int64_t)b * a.chunks + c) * a.hv + h) * a.dk * a.dv;
    const float* dstate = a.w.dstate + at * a.dk * a.dvp;
    const float* before = c ? dstate - (int64_t)a.dk * a.dvp : a.dh0 + bh * a.dk * a.dv;
    const int ldb = c ? a.dvp : a.dv;
    const float* zs = a.w.z + at * kChunk * a.dvp;
    const Range vs = rows_range<T>(a.v, b, h, c * kChunk, a.t, a.dv), dys = rows_range<T>(a.dy, b, h, c * kChunk, a.t, a.dv);
    const auto fetch = [&](int v0, Slice& x) {
      load_state(states, v0, a.dv, x.s);
      load_state(dstate, v0, a.dvp, x.ds);
      load_state(before, v0, ldb, x.before);
      const int col = v0 + 16 * half + m;
      const uint32_t ld = row_bytes<T>(a.v), at_v = col < a.dv ? own * ld + (uint32_t)col * (uint32_t)sizeof(T) : kNowhere;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x.z[i] = load_at<float>(zs + (int64_t)i * a.dvp + v0, (uint32_t)(own * a.dvp + 16 * half + m) * 4u);
        x.v[i] = vs.load<T>(at_v + i * ld);
      }
      const uint32_t dy_row = row() * row_bytes<T>(a.dy);
      if (a.vec_dy) {
        x.dy.load(dys, dy_row, v0 + 8 * q4, a.dv);
      } else {
        T e8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          e8[e] = dys.load<T>(v0 + 8 * q4 + e < a.dv ? dy_row + (uint32_t)(v0 + 8 * q4 + e) * (uint32_t)sizeof(T) : kNowhere);
        __builtin_memcpy(x.dy.w, e8, sizeof(e8));
      }
    };
    Slice x;
    fetch(0, x);
    __syncthreads();  // what is read of the head before
    for (int i = tid; i < 3 * kChunk; i += kT) s.gates[i] = a.w.rows[at * 4 * kChunk + i];
    if (tid < kChunk) {
      s.sums[tid] = a.w.sums[at * kChunk + tid];
      s.seq[tid] = a.w.seq[at * kChunk + tid];
    }
    if (tid < 2) s.bad[tid] = 0;
    k.put(s.rows);
    bool wild = !k.finite() || !q.finite();
    wild = __syncthreads_or(wild);
    const f32x4_t enter = *(const f32x4_t*)(s.gates + own), leave = *(const f32x4_t*)(s.gates + kChunk + own);
    const f32x4_t beta = *(const f32x4_t*)(s.gates + 2 * kChunk + own);
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    f32x4_t dkr[DT], dkc[DT], dp[2] = {zero, zero}, dl[2] = {zero, zero}, db = zero, dxv = zero;
    float dot = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t) dq[t] = dkr[t] = dkc[t] = zero;
#pragma clang loop unroll(disable)
    for (int v0 = 0; v0 < a.dvp; v0 += kCols) {
      renew();
      if (v0) __syncthreads();  // what is read of the slice before
      within(x.s, v0, a.dv);
      within(x.ds, v0, a.dvp);
      put_state<kParts>(s.s, x.s);
      put_state<GP>(s.ds, x.ds);
      if (each || tid < DK * kCols / 4)
#pragma unroll
        for (int n = 0; n < held; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = fmaf(x.s[n][e], x.before[n][e], dot);  // S is zero outside
      // r and dx; rows past T and columns past Dv hold nothing
      f32x4_t r, z = x.z, dx;
      float e8[8];
      x.dy.get(e8);
#pragma unroll
      for (int e = 0; e < 8; ++e) e8[e] = c * kChunk + row() < a.t ? e8[e] : 0.f;
      const Parts<NP> yp = split<NP>(e8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = c * kChunk + own + i < a.t ? to_f32(x.v[i]) : 0.f;
        dx[i] = beta[i] * z[i];
        dxv[i] = fmaf(dx[i], r[i], dxv[i]);
      }
      if (v0 + kCols < a.dvp) fetch(v0 + kCols, x);
      put_rows<GP>(s.dx, dx);
      __syncthreads();
      renew();
      {
        f32x4_t ks = zero, more = zero;
#pragma unroll
        for (int e = 0; e < KS; ++e) {
          const auto kp = natural<NP>(s.rows + row() * RowsAt<DK>::stride + 32 * e + 8 * q4, RowsAt<DK>::part);
          const auto sp = transposed<kParts>(s.s + (32 * e + 8 * q4 + m / 4) * kSlice + 16 * half + 4 * (m % 4), kSlice, DK * kSlice);
          (e & 1 ? more : ks) = mma(kp, sp, e & 1 ? more : ks);
          if (e & 1) __builtin_amdgcn_sched_barrier(0);
        }
        bf164_t o[kParts];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[i] -= times(enter[i], ks[i] + more[i]);
          __bf16 w[kParts];
          split_one<kParts>(beta[i] * r[i], w);
#pragma unroll
          for (int n = 0; n < kParts; ++n) o[n][i] = w[n];
        }
#pragma unroll
        for (int n = 0; n < kParts; ++n)
          *(bf164_t*)(s.br + (half * kParts + n) * F::Rows::part + m * F::Rows::ld + own) = o[n];
      }
      __syncthreads();
      renew();
      f32x4_t xs;
      bool masked = false;
#pragma clang loop unroll(disable)
      for (;;) {
        int hi = kChunk;
#pragma clang loop unroll(disable)
        do {
          int lo = 0;
          if (masked)
            for (lo = hi - 1; lo > 0 && s.seq[lo] == s.seq[lo - 1];) --lo;
          f32x4_t n = r, more = zero;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (e <= wave / 2) {
              Parts<kParts> hp = solve[e];
              auto bp = natural<kParts>(s.br + half * kParts * F::Rows::part + m * F::Rows::ld + 32 * e + 8 * q4, F::Rows::part);
              if (masked) keep(hp, 32 * e + 8 * q4, lo, hi), keep(bp, 32 * e + 8 * q4, lo, hi);
              (e ? more : n) = mma(hp, bp, e ? more : n);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (own + i >= lo && own + i < hi) xs[i] = n[i] + more[i];
          hi = lo;
        } while (hi > 0);
        float test = 0.f;
        f32x4_t u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i] = beta[i] * xs[i];
          test = fmaf(xs[i], 0.f, test);
        }
        put_rows<kParts>(s.u, u);
        if (__any(test != 0.f)) s.bad[turn & 1] = 1;  // NaN
        __syncthreads();
        const bool bad = s.bad[turn & 1];
        if (tid == 0) s.bad[~turn & 1] = 0;
        ++turn;
        if (masked || !bad) break;
        masked = true;
        __syncthreads();  // the flags, and u, are read before they are written again
      }
      renew();
#pragma unroll
      for (int i = 0; i < 4; ++i) db[i] = fmaf(xs[i], z[i], db[i]);
      const auto up = slice<kParts>(s.u, row(), kChunk);
      const auto xp = slice<GP>(s.dx, row(), kChunk);
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const int d = 16 * (half * DT + t) + m;
        const auto sp = slice<kParts>(s.s, d, DK);
        const auto dsp = slice<GP>(s.ds, d, DK);
        dq[t] = mma(yp, sp, dq[t]);
        dkr[t] = mma_first<GP>(xp, sp, dkr[t]);
        dkc[t] = mma_first<GP>(up, dsp, dkc[t]);
        __builtin_amdgcn_sched_barrier(0);  // or the operands of all tiles are held at once
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (half + 2 * n <= wave) {
          const auto uj = slice<kParts>(s.u, 16 * (half + 2 * n) + m, kChunk);
          dp[n] = mma(yp, uj, dp[n]);
          dl[n] = mma_first<GP>(xp, uj, dl[n]);
        }
    }
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dq[t][r] = times(enter[r], a.scale * dq[t][r]);
        dk[t][r] = times(leave[r], dkc[t][r]) - times(enter[r], dkr[t][r]);
      }
    for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o);
    if (lane == 0) s.a[4 * half + wave] = dot;
    renew();
    __syncthreads();  // the slices are read: their room is the matrices' now
    put_matrix<true, kParts>(s.p, dp, a.scale);
    put_matrix<false, GP>(s.l, dl, -1.f);
    __syncthreads();
    renew();
    add<false, kParts>(s.p, dq, wild);
    renew();
    add<false, GP>(s.l, dk, wild);
    renew();
    add<true, GP>(s.l, dk, wild);
    renew();
    __syncthreads();
    q.put(s.rows);
    __syncthreads();
    renew();
    add<true, GP>(s.p, dk, wild);
    renew();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float g = 0.f;
#pragma unroll
      for (int t = 0; t < DT; ++t) g = fmaf(value(s.rows, own + r, 16 * (half * DT + t) + m), dq[t][r], g);
      const float qdq = over_lanes(g), xv = over_lanes(dxv[r]), dbr = over_lanes(db[r]);
      if (m == 0) {
        s.red[half][own + r][0] = qdq;
        s.red[half][own + r][1] = xv;
        s.red[half][own + r][2] = dbr;
      }
    }
    __syncthreads();
    if (tid < kChunk) {
      const int mine = s.seq[lane], t = c * kChunk + lane;
      double sum = ((double)s.red[0][lane][1] + s.red[1][lane][1]) - ((double)s.red[0][lane][0] + s.red[1][lane][0]), g = 0;
      if (mine == 0)
        for (int w = 0; w < kT / 64; ++w) g += s.a[w];
      // the rows before, of the same sequence
      for (int o = 1; o < 64; o <<= 1) {
        const double p = __shfl_up(sum, o);
        const int of = __shfl_up(mine, o);
        if (lane >= o && of == mine) sum += p;
      }
      const double p = __shfl_up(sum, 1);
      const int of = __shfl_up(mine, 1);
      if (lane > 0 && of == mine) g += p;
      if (t < a.t) {
        const int64_t to = ((int64_t)b * a.t + t) * a.hv + h;
        a.dlog_decay[to] = (float)g;
        a.dbeta[to] = s.red[0][lane][2] + s.red[1][lane][2];
      }
    }
  }
};

template <typename T, int DK>
__global__ __launch_bounds__(kT, 1) void delta_grad_kernel(DeltaArgs a) {
  typedef Grad<T, DK> F;
  __shared__ __attribute__((aligned(16))) typename F::Lds s;
  // neighbouring chunks on one die: each reads the gradient of a state that its neighbour reads too
  const int id = convfwd::xcd_tile(blockIdx.x, gridDim.x);
  const int c = id % a.chunks, hk = id / a.chunks % a.hk, b = id / a.chunks / a.hk;
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
    hipLaunchKernelGGL((delta_grad_kernel<T, decltype(dk)::value>), dim3(a.b * a.hk * a.chunks), dim3(kT), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace convdelta
