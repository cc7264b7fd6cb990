// k_delta_prep.hip -- gated delta rule, what a chunk of 64 rows holds that no
// state enters: the decays, H and the decayed q k^T (see delta_device.h), one
// workgroup a chunk and value head, all chunks at once.
//
// 4096 chunks and heads of 128, bf16: 75 us (3 TB/s of operands and rows); bound by the
// chain inside a workgroup (16 rows substituted one after the other, then six rounds of
// 16 x 16 blocks on the fp32 matrix units: 191 us with all 64 rows substituted), four
// workgroups a CU.  H and its transpose are made for each direction and not kept: 37 KB a
// chunk and head written and read again would cost what making them does.
#include "delta_team.h"

namespace convdelta {

namespace {

constexpr int kT = 256, kLd = kChunk + 1, kLdX = 17;

// Where row i, columns j0 .. + 7 (or, UP, column i, rows j0 .. + 7) of a lower triangle start: in place, or (H) in the
// block across the diagonal.
template <bool UP, bool H>
__device__ __forceinline__ const float* place(const float* m, int i, int j0) {
  const int bi = i / 16, bj = j0 / 16;
  if (H && bi != bj) return UP ? m + (16 * bi + j0 % 16) * kLd + 16 * bj + i % 16 : m + (16 * bj + i % 16) * kLd + 16 * bi + j0 % 16;
  return UP ? m + j0 * kLd + i : m + i * kLd + j0;
}

// Writes a 64x64 lower triangle of LDS as operands of a product with its rows (or, UP, its columns) as rows, in N parts.
template <bool UP, bool H, int N>
__device__ __forceinline__ void put_matrix(const float* m, char* to) {
  const int wave = wave_id(), lane = threadIdx.x % 64, q = lane / 16;
  for (int f = wave; f < kTri; f += kT / 64) {
    const int row = 16 * (UP ? up_t(f) : low_t(f)) + lane % 16, k0 = 32 * (UP ? up_s(f) : low_s(f)) + 8 * q;
    const float* from = place<UP, H>(m, row, k0);
    const bool none = UP ? k0 / 16 < row / 16 : k0 / 16 > row / 16;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = none ? 0.f : from[UP ? e * kLd : e];
    const Parts<N> p = split<N>(x);
#pragma unroll
    for (int n = 0; n < N; ++n) *(bf168_t*)(to + (f * kParts + n) * kFrag + lane * 16) = p.p[n];
  }
}

// D += A B for 16x16 blocks in LDS, A's rows kLd apart and its columns scaled (a zero of A stays zero, whatever the
// scale): fp32 matrix instructions, in each of which lane l supplies A[l % 16][k] and B[k][l % 16] for k = 4 step + l / 16.
__device__ __forceinline__ f32x4_t block_product(const float* a, const float* scale, const float* b, int ldb, f32x4_t acc) {
  const int m = threadIdx.x % 16, q4 = threadIdx.x % 64 / 16;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(times(a[m * kLd + 4 * k + q4], scale[4 * k + q4]), b[(4 * k + q4) * ldb + m],
                                               acc, 0, 0, 0);
  return acc;
}

// L (64x64, strictly lower, the rest zero) becomes H = -(I + L beta)^-1 L, whose rows are
// H_i = -L_i - sum over k < i of L_ik beta_k H_k.  Blocks of 16: the diagonal ones row by row, each by a wave,
// then the ones at distance 1, 2 and 3 below them:
//   X_ij = -L_ij - sum over j <= k < i of L_ik beta_k H_kj,  H_ij = X_ij + H_ii beta_i X_ij.
// The diagonal blocks take L's place; the others, whose L is needed to the end, go across the diagonal.  `x` is room
// for the X of one distance.
__device__ __forceinline__ void invert(float* l, const float* beta, float* x) {
  const int wave = wave_id(), lane = threadIdx.x % 64, m = lane % 16, q4 = lane / 16;
  {
    // column m of the diagonal block; what lies on and above the diagonal stays zero, whatever a row holds
    float* d = l + 16 * wave * (kLd + 1);
    const float* bt = beta + 16 * wave;
    float bh[16], hc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[2] = {-d[i * kLd + m], 0.f};
#pragma unroll
      for (int k = 0; k < i; ++k) s[k & 1] = fmaf(-d[i * kLd + k], bh[k], s[k & 1]);
      hc[i] = m < i ? s[0] + s[1] : 0.f;
      bh[i] = m < i ? bt[i] * hc[i] : 0.f;
    }
    if (q4 == 0)  // the four quarters of the wave compute the same
#pragma unroll
      for (int i = 0; i < 16; ++i) d[i * kLd + m] = hc[i];
  }
#pragma unroll
  for (int far = 1; far < 4; ++far) {
    __syncthreads();
    const int bi = wave + far, bj = wave;  // this wave's block, where there is one
    const float* from = l + 16 * bi * kLd + 16 * bj;
    float* to = l + 16 * bj * kLd + 16 * bi;
    f32x4_t xs;
    if (bi < 4) {
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < far; ++k)
        acc = block_product(from + 16 * k, beta + 16 * (bj + k), k ? to - 16 * (far - k) : l + 16 * bj * (kLd + 1), kLd, acc);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        xs[r] = -from[(4 * q4 + r) * kLd + m] - acc[r];
        x[(16 * wave + 4 * q4 + r) * kLdX + m] = xs[r];
      }
    }
    __syncthreads();
    if (bi < 4) {
      xs = block_product(l + 16 * bi * (kLd + 1), beta + 16 * bi, x + 16 * wave * kLdX, kLdX, xs);
#pragma unroll
      for (int r = 0; r < 4; ++r) to[(4 * q4 + r) * kLd + m] = xs[r];
    }
  }
  __syncthreads();
}

template <typename T, int DK>
struct PrepLds {
  union {
    __bf16 k[InParts<T>::n * RowsAt<DK>::part];
    struct {
      float low[kChunk * kLd], read[kChunk * kLd];
    };
  };
  float x[3 * 16 * kLdX];
  double sums[kChunk];
  float beta[kChunk];
  int seq[kChunk];
};

template <typename T, int DK>
__global__ __launch_bounds__(kT) void delta_prep_kernel(DeltaArgs a, int backward) {
  constexpr int NP = InParts<T>::n, KS = DK / 32;
  typedef Team<T, DK, 1> F;
  __shared__ __attribute__((aligned(16))) PrepLds<T, DK> s;
  const int c = blockIdx.x % a.chunks, t0 = c * kChunk;
  const F f(a, blockIdx.x / a.chunks, 0);
  const int wave = wave_id(), lane = f.lane, m = f.m, q4 = f.q4;
  const int64_t at = chunk_index(a, f.bh, c);
  Raw8<T> k[KS], q[KS];
  f.load_rows(a.k, c, k);
  f.load_rows(a.q, c, q);
  // rows past T decay nothing and write nothing
  const int t = t0 + lane;
  const bool in = wave == 0 && t < a.t;
  const int64_t row = ((int64_t)f.b * a.t + t) * a.hv + f.h;
  const float bt = in ? a.beta[row] : 0.f;
  const float g = in ? a.log_decay[row] : 0.f;
  int start = in && a.starts ? a.starts[(int64_t)f.b * a.t + t] != 0 : 0;
  f.put_rows(s.k, k);
  __syncthreads();
  if (wave == 0) {
    // running sums over the rows, a lane a row (this wave has the fewest products)
    // a decay that is zero in fp32 drops the state: its row begins a sequence too, and its gradient is zero
    const float step = start ? 0.f : expf(g);
    start |= step == 0.f;
    // what is at a start acts on nothing, whatever it is
    double sum = start ? 0.f : g;
    int n = start;
    for (int o = 1; o < 64; o <<= 1) {
      const int p = __shfl_up(n, o);
      if (lane >= o) n += p;
    }
    // within a sequence only: what is not finite must not reach the next one's differences
    for (int o = 1; o < 64; o <<= 1) {
      const double p = __shfl_up(sum, o);
      const int pn = __shfl_up(n, o);
      if (lane >= o && pn == n) sum += p;
    }
    const double all = __shfl(sum, 63);
    const int last = __shfl(n, 63);
    s.sums[lane] = sum;
    s.seq[lane] = n;
    s.beta[lane] = bt;
    float* rows = a.w.rows + at * 4 * kChunk;
    rows[lane] = n == 0 ? expf((float)sum) : 0.f;
    rows[kChunk + lane] = n == last ? expf((float)(all - sum)) : 0.f;
    rows[2 * kChunk + lane] = bt;
    rows[3 * kChunk + lane] = step;
    if (backward) {
      a.w.sums[at * kChunk + lane] = sum;
      a.w.seq[at * kChunk + lane] = n;
    }
  }
  // this wave's rows of k k^T and q k^T
  f32x4_t kk[4], qk[4];
#pragma unroll
  for (int tj = 0; tj < 4; ++tj) {
    kk[tj] = qk[tj] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (tj <= wave)
#pragma unroll
      for (int e = 0; e < KS; ++e) {
        const auto kb = natural<NP>(s.k + (16 * tj + m) * RowsAt<DK>::stride + 32 * e + 8 * q4, RowsAt<DK>::part);
        kk[tj] = mma(f.rows_of(k, e), kb, kk[tj]);
        qk[tj] = mma(f.rows_of(q, e), kb, qk[tj]);
      }
  }
  __syncthreads();  // k is read: its room is the matrices' now
  double si[4];
  int ni[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) si[r] = s.sums[f.row() + r], ni[r] = s.seq[f.row() + r];
#pragma unroll
  for (int tj = 0; tj < 4; ++tj) {
    const int j = 16 * tj + m, nj = s.seq[j];
    const double sj = s.sums[j];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = f.row() + r;
      const bool same = j <= i && ni[r] == nj;
      const float d = expf((float)(si[r] - sj));  // no branch: what is not wanted is selected away
      s.low[i * kLd + j] = same && j < i ? d * kk[tj][r] : 0.f;
      s.read[i * kLd + j] = same ? d * qk[tj][r] : 0.f;
    }
  }
  __syncthreads();
  invert(s.low, s.beta, s.x);
  if (!backward) {
    put_matrix<false, true, kParts>(s.low, a.w.solve + at * kMatrix);
    put_matrix<false, false, kParts>(s.read, a.w.read + at * kMatrix);
  } else {
    put_matrix<true, true, kParts>(s.low, a.w.solve_t + at * kMatrix);
    put_matrix<true, false, kParts>(s.read, a.w.read_t + at * kMatrix);
  }
}

// q and k of other alignments or sizes, copied to rows of dkp elements, the spare ones zero.
template <typename T>
__global__ __launch_bounds__(kT) void delta_pack_kernel(DeltaArgs a, Heads q, Heads k, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kT + threadIdx.x;
  if (i >= n) return;
  const int pieces = a.dkp / 8, d0 = (int)(i % pieces) * 8;
  const int64_t r = i / pieces, h = r % a.hk, t = r / a.hk % a.t, b = r / a.hk / a.t;
  const T *fq = (const T*)q.p + b * q.sb + t * q.st + h * q.sh, *fk = (const T*)k.p + b * k.sb + t * k.st + h * k.sh;
  T vq[8], vk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    vq[e] = d0 + e < a.dk ? fq[d0 + e] : (T)0.f;
    vk[e] = d0 + e < a.dk ? fk[d0 + e] : (T)0.f;
  }
  const Heads to = packed_rows(nullptr, a.t, a.hk, a.dkp);
  const int64_t at = b * to.sb + t * to.st + h * to.sh + d0;
  __builtin_memcpy(__builtin_assume_aligned((T*)a.w.q + at, 16), vq, sizeof(vq));
  __builtin_memcpy(__builtin_assume_aligned((T*)a.w.k + at, 16), vk, sizeof(vk));
}

}  // namespace

hipError_t launch_delta_pack(const DeltaArgs& a, const Heads& q, const Heads& k, hipStream_t s) {
  const int64_t n = (int64_t)a.b * a.t * a.hk * (a.dkp / 8);
  return for_type(a.dtype, [&](auto t) {
    hipLaunchKernelGGL((delta_pack_kernel<decltype(t)>), dim3((unsigned)((n + kT - 1) / kT)), dim3(kT), 0, s, a, q, k, n);
    return hipGetLastError();
  });
}

hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t s) {
  return for_type(a.dtype, [&](auto t) {
    return for_dk(a.dk, [&](auto dk) {
      hipLaunchKernelGGL((delta_prep_kernel<decltype(t), decltype(dk)::value>), dim3(a.b * a.hv * a.chunks), dim3(kT), 0, s,
                         a, (int)backward);
      return hipGetLastError();
    });
  });
}

}  // namespace convdelta
