// delta_grad.h -- gated delta rule, the gradients that add over all columns of v: one
// workgroup a chunk and key head, all chunks at once.  With u = beta x, dx = beta z,
// S the state before the chunk and dS the gradient of the one after it,
//
//   dP = scale * D * (dy u^T) (j <= i),  dL = -D * (dx u^T) (j < i)
//   dq = scale * enter * (dy S^T) + dP k
//   dk = [-enter * (dx S^T) + dL k] + [leave * (u dS^T) + dP^T q + dL^T k]
//
// and, with the two brackets dk_row and dk_col, the gradient of the sums of log decays
// is q.dq + k.dk_row - k.dk_col, at the last row with enter_last <S, dS> + sum of
// leave * (u dS^T).k besides; dlog_decay is its running sum from the end of each sequence.
// Included by one source for each type.
#include "delta_device.h"

namespace convdelta {

namespace {

constexpr int kT = 256, kCols = 32, kSlice = kCols + 8, kLdM = kChunk + 8;

template <typename T, int DK>
struct GradLds {
  static constexpr int NP = InParts<T>::n;
  __bf16 k[NP * RowsAt<DK>::part], q[NP * RowsAt<DK>::part];
  union {
    struct {
      __bf16 s[kParts * DK * kSlice];     // 32 columns of a state, rows d
      __bf16 u[kParts * kChunk * kSlice]; // and of u, rows j
    };
    __bf16 m[kParts * kChunk * kLdM];     // dP or dL
  };
  float rows[4 * kChunk], dg[kChunk], sum[kT / 64][2];
  double sums[kChunk];
  int seq[kChunk];
};

template <typename T, int DK>
struct Grad {
  static constexpr int NP = InParts<T>::n, DT = DK / 16, kSp = DK * kCols / 4 / kT;  // pieces of 4 floats a thread
  typedef GradLds<T, DK> Lds;
  const DeltaArgs& a;
  Lds& s;
  int wave, lane, m, q4, b, c, row, own;  // row: the lane's row as an operand; own: its first row of accumulators

  __device__ __forceinline__ Grad(const DeltaArgs& a_, Lds& s_, int b_, int c_) : a(a_), s(s_), b(b_), c(c_) {
    wave = wave_id();
    lane = threadIdx.x % 64;
    m = lane % 16;
    q4 = lane / 16;
    row = 16 * wave + m;
    own = 16 * wave + 4 * q4;
  }

  // 32 columns of a (Dk, ld) state, of which `width` are there, as parts into LDS
  __device__ __forceinline__ void load_state(const float* from, int v0, int ld, int width, bool whole, f32x4_t (&x)[kSp]) const {
#pragma unroll
    for (int k = 0; k < kSp; ++k) {
      const int i = threadIdx.x + k * kT, d = i / (kCols / 4), v = v0 + i % (kCols / 4) * 4;
      const float* p = from + (int64_t)d * ld + v;
      if (d < a.dk && whole && v < width) {
        x[k] = *(const f32x4_t*)p;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] = d < a.dk && v + e < width ? p[e] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void put_state(const f32x4_t (&x)[kSp]) const {
#pragma unroll
    for (int k = 0; k < kSp; ++k) {
      const int i = threadIdx.x + k * kT, d = i / (kCols / 4), v = i % (kCols / 4) * 4;
      bf164_t o[kParts];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        __bf16 w[kParts];
        split_one<kParts>(x[k][e], w);
#pragma unroll
        for (int n = 0; n < kParts; ++n) o[n][e] = w[n];
      }
#pragma unroll
      for (int n = 0; n < kParts; ++n) *(bf164_t*)(s.s + (n * DK + d) * kSlice + v) = o[n];
    }
  }

  __device__ __forceinline__ float value(const __bf16* x, int r, int d) const {
    float v = 0.f;
#pragma unroll
    for (int n = NP - 1; n >= 0; --n) v += (float)x[n * RowsAt<DK>::part + r * RowsAt<DK>::stride + d];
    return v;
  }

  // out (own rows, all d) += M k or M^T k with M in LDS; MASKED: over the rows [lo, hi), which are the only ones added to
  template <bool UP, bool MASKED>
  __device__ __forceinline__ void add_range(const __bf16* x, f32x4_t (&out)[DT], int lo, int hi) const {
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      f32x4_t n = out[t];
      if (MASKED) n = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // a triangle: rows of this wave's tile hold nothing in the other half
        if (UP ? k < wave / 2 : k > wave / 2) continue;
        const Parts<kParts> am = UP ? transposed<kParts>(s.m + (32 * k + 8 * q4 + m / 4) * kLdM + 16 * wave + 4 * (m % 4), kLdM, kChunk * kLdM)
                                    : natural<kParts>(s.m + row * kLdM + 32 * k + 8 * q4, kChunk * kLdM);
        Parts<NP> bm = transposed<NP>(x + (32 * k + 8 * q4 + m / 4) * RowsAt<DK>::stride + 16 * t + 4 * (m % 4), RowsAt<DK>::stride,
                                      RowsAt<DK>::part);
        if (MASKED) keep(bm, 32 * k + 8 * q4, lo, hi);
        n = mma(am, bm, n);
      }
      if (!MASKED) out[t] = n;
      if (MASKED)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (own + r >= lo && own + r < hi) out[t][r] += n[r];
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  template <bool UP>
  __device__ __forceinline__ void add(const __bf16* x, f32x4_t (&out)[DT], bool wild) const {
    if (!wild) return add_range<UP, false>(x, out, 0, kChunk);
    int hi = kChunk;
#pragma clang loop unroll(disable)
    for (int lo = kChunk - 1; lo >= 0; --lo)
      if (lo == 0 || s.seq[lo] != s.seq[lo - 1]) {
        add_range<UP, true>(x, out, lo, hi);
        hi = lo;
      }
  }

  // M = factor * D * acc below (and, EDGE, on) the diagonal, as parts into LDS
  template <bool EDGE>
  __device__ __forceinline__ void put_matrix(const f32x4_t (&acc)[4], float factor) const {
#pragma unroll
    for (int tj = 0; tj < 4; ++tj) {
      const int j = 16 * tj + m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = own + r;
        const bool in = (EDGE ? j <= i : j < i) && s.seq[i] == s.seq[j];
        const float x = in ? factor * expf((float)(s.sums[i] - s.sums[j])) * acc[tj][r] : 0.f;
        __bf16 w[kParts];
        split_one<kParts>(x, w);
#pragma unroll
        for (int n = 0; n < kParts; ++n) s.m[(n * kChunk + i) * kLdM + j] = w[n];
      }
    }
  }

  __device__ __forceinline__ float over_lanes(float v) const {
    for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o);
    return v;
  }

  // The gradients of one value head; its share of dq and dk.
  __device__ __forceinline__ void head(int h, bool wild, f32x4_t (&dq)[DT], f32x4_t (&dk)[DT]) const {
    const int64_t bh = (int64_t)b * a.hv + h, at = bh * a.chunks + c;
    __syncthreads();  // what is read of the head before
    for (int i = threadIdx.x; i < 4 * kChunk; i += kT) s.rows[i] = a.w.rows[at * 4 * kChunk + i];
    if (threadIdx.x < kChunk) {
      s.sums[threadIdx.x] = a.w.sums[at * kChunk + threadIdx.x];
      s.seq[threadIdx.x] = a.w.seq[at * kChunk + threadIdx.x];
    }
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    f32x4_t dkr[DT], dkc[DT], dp[4], dl[4];
#pragma unroll
    for (int t = 0; t < DT; ++t) dq[t] = dkr[t] = dkc[t] = zero;
#pragma unroll
    for (int t = 0; t < 4; ++t) dp[t] = dl[t] = zero;
    const float* states = a.states_in + (((int64_t)b * a.chunks + c) * a.hv + h) * a.dk * a.dv;
    const float* dstate = a.w.dstate + at * a.dk * a.dvp;
    const float *xr = a.w.x + (at * kChunk + row) * a.dvp, *zr = a.w.z + (at * kChunk + row) * a.dvp;
    const T* dy = (const T*)a.dy.p + b * a.dy.sb + (int64_t)min(c * kChunk + row, a.t - 1) * a.dy.st + h * a.dy.sh;
    const bool in = c * kChunk + row < a.t, whole = a.dv % 4 == 0;
    float dot = 0.f, db = 0.f;
    __syncthreads();
    const float beta = s.rows[2 * kChunk + row];
    for (int v0 = 0; v0 < a.dvp; v0 += kCols) {
      f32x4_t st[kSp], ds[kSp];
      load_state(states, v0, a.dv, a.dv, whole, st);
      load_state(dstate, v0, a.dvp, a.dvp, true, ds);
      const int v = v0 + 8 * q4;
      float u[8], dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = xr[v + e], z = zr[v + e];
        u[e] = beta * x;
        dx[e] = beta * z;
        db = fmaf(x, z, db);
      }
      float yv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) yv[e] = in && v + e < a.dv ? to_f32(dy[v + e]) : 0.f;
      const Parts<NP> yp = split<NP>(yv);
      const Parts<kParts> up = split<kParts>(u), xp = split<kParts>(dx);
      __syncthreads();  // what is read of the slice before
      put_state(st);
#pragma unroll
      for (int n = 0; n < kParts; ++n) *(bf168_t*)(s.u + (n * kChunk + row) * kSlice + 8 * q4) = up.p[n];
      __syncthreads();
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const auto sp = natural<kParts>(s.s + (16 * t + m) * kSlice + 8 * q4, DK * kSlice);
        dq[t] = mma(yp, sp, dq[t]);
        dkr[t] = mma(xp, sp, dkr[t]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int tj = 0; tj < 4; ++tj)
        if (tj <= wave) {
          const auto uj = natural<kParts>(s.u + (16 * tj + m) * kSlice + 8 * q4, kChunk * kSlice);
          dp[tj] = mma(yp, uj, dp[tj]);
          dl[tj] = mma(xp, uj, dl[tj]);
        }
      __syncthreads();
      put_state(ds);
#pragma unroll
      for (int k = 0; k < kSp; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = fmaf(st[k][e], ds[k][e], dot);
      __syncthreads();
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const auto sp = natural<kParts>(s.s + (16 * t + m) * kSlice + 8 * q4, DK * kSlice);
        dkc[t] = mma(up, sp, dkc[t]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    db += __shfl_xor(db, 16);
    db += __shfl_xor(db, 32);
    if (q4 == 0 && in) a.dbeta[((int64_t)b * a.t + c * kChunk + row) * a.hv + h] = db;
    // the decays of the rows, and what the last row's sum gets besides
    const f32x4_t enter = *(const f32x4_t*)(s.rows + own), leave = *(const f32x4_t*)(s.rows + kChunk + own);
    float more = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dq[t][r] = times(enter[r], a.scale * dq[t][r]);
        dkr[t][r] = -times(enter[r], dkr[t][r]);
        dkc[t][r] = times(leave[r], dkc[t][r]);
        if (leave[r] != 0.f) more = fmaf(value(s.k, own + r, 16 * t + m), dkc[t][r], more);
      }
    for (int o = 1; o < 64; o <<= 1) {
      dot += __shfl_xor(dot, o);
      more += __shfl_xor(more, o);
    }
    if (lane == 0) {
      s.sum[wave][0] = dot;
      s.sum[wave][1] = more;
    }
    __syncthreads();  // the slices are read: their room is the matrices' now
    put_matrix<true>(dp, a.scale);
    __syncthreads();
    add<false>(s.k, dq, wild);
    add<true>(s.q, dkc, wild);
    __syncthreads();
    put_matrix<false>(dl, -1.f);
    __syncthreads();
    add<false>(s.k, dkr, wild);
    add<true>(s.k, dkc, wild);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float g = 0.f;
#pragma unroll
      for (int t = 0; t < DT; ++t)
        g += value(s.q, own + r, 16 * t + m) * dq[t][r] + value(s.k, own + r, 16 * t + m) * (dkr[t][r] - dkc[t][r]);
      g = over_lanes(g);
      if (m == 0) s.dg[own + r] = g;
    }
#pragma unroll
    for (int t = 0; t < DT; ++t) dk[t] = dkr[t] + dkc[t];
    __syncthreads();
    if (wave == 0) {
      const float stay = s.rows[kChunk - 1];
      double tail = 0;
      for (int w = 0; w < kT / 64; ++w) tail += (double)times(stay, s.sum[w][0]) + s.sum[w][1];
      const int mine = s.seq[lane];
      double g = mine == s.seq[kChunk - 1] ? tail : 0.0;
      for (int j = kChunk - 1; j >= 0; --j)
        if (j >= lane && s.seq[j] == mine) g += s.dg[j];
      // the decay of a row at a start acts on nothing
      if (mine != (lane ? s.seq[lane - 1] : 0)) g = 0;
      const int t = c * kChunk + lane;
      if (t < a.t) a.dlog_decay[((int64_t)b * a.t + t) * a.hv + h] = (float)g;
    }
  }
};

template <typename T, int DK>
__global__ __launch_bounds__(kT) void delta_grad_kernel(DeltaArgs a) {
  typedef Grad<T, DK> F;
  __shared__ __attribute__((aligned(16))) typename F::Lds s;
  const int c = blockIdx.x % a.chunks, hk = blockIdx.x / a.chunks % a.hk, b = blockIdx.x / a.chunks / a.hk;
  F f(a, s, b, c);
  bool wild = false;
  {
    Rows64<T, DK, kT> k, q;
    k.load(a.k, b, hk, c * kChunk, a.t, a.dkp);
    q.load(a.q, b, hk, c * kChunk, a.t, a.dkp);
#pragma unroll
    for (int i = 0; i < Rows64<T, DK, kT>::each; ++i) {
      float x[8], y[8];
      k.p[i].get(x, true);
      q.p[i].get(y, true);
#pragma unroll
      for (int e = 0; e < 8; ++e) wild = wild || !finite(x[e]) || !finite(y[e]);
    }
    k.put(s.k, a.dkp);
    q.put(s.q, a.dkp);
  }
  wild = __syncthreads_or(wild);
  const int share = a.hv / a.hk;
  f32x4_t dq[F::DT], dk[F::DT], sq[F::DT], sk[F::DT];
  for (int n = 0; n < share; ++n) {
    f.head(hk * share + n, wild, dq, dk);
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
      const int row = f.own + r, d = 16 * t + f.m;
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
