// k_delta_prep.hip -- gated delta rule, what a chunk of 64 rows holds that no
// state enters: the decays, H and the decayed q k^T (see delta_device.h), one
// workgroup a chunk and value head, all chunks at once.
#include "delta_device.h"

namespace convdelta {

namespace {

constexpr int kT = 256, kLd = kChunk + 1;

// Writes a 64x64 matrix of LDS as operands of a product with its rows (or, UP, its columns) as rows.
template <bool UP>
__device__ __forceinline__ void put_matrix(const float* m, char* to) {
  const int wave = wave_id(), lane = threadIdx.x % 64, q = lane / 16;
  for (int f = wave; f < kTri; f += kT / 64) {
    const int row = 16 * (UP ? up_t(f) : low_t(f)) + lane % 16, k0 = 32 * (UP ? up_s(f) : low_s(f)) + 8 * q;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = UP ? m[(k0 + e) * kLd + row] : m[row * kLd + k0 + e];
    const Parts<kParts> p = split<kParts>(x);
#pragma unroll
    for (int n = 0; n < kParts; ++n) *(bf168_t*)(to + (f * kParts + n) * kFrag + lane * 16) = p.p[n];
  }
}

template <typename T, int DK>
__global__ __launch_bounds__(kT) void delta_prep_kernel(DeltaArgs a, int backward) {
  constexpr int NP = InParts<T>::n;
  __shared__ __attribute__((aligned(16))) __bf16 ks[NP * RowsAt<DK>::part], qs[NP * RowsAt<DK>::part];
  __shared__ float low[kChunk * kLd], read[kChunk * kLd];
  __shared__ double sums[kChunk];
  __shared__ float beta[kChunk];
  __shared__ int seq[kChunk];
  const int c = blockIdx.x % a.chunks, bh = blockIdx.x / a.chunks, b = bh / a.hv, h = bh % a.hv, t0 = c * kChunk;
  const int wave = wave_id(), lane = threadIdx.x % 64;
  const int64_t at = chunk_index(a, bh, c);
  {
    Rows64<T, DK, kT> k, q;
    k.load(a.k, b, h / (a.hv / a.hk), t0, a.t, a.dkp);
    q.load(a.q, b, h / (a.hv / a.hk), t0, a.t, a.dkp);
    if (wave == 0) {
      // running sums over the rows, a lane a row; rows past T decay nothing and write nothing
      const int t = t0 + lane;
      const bool in = t < a.t;
      const int64_t row = ((int64_t)b * a.t + t) * a.hv + h;
      const float bt = in ? a.beta[row] : 0.f;
      // a decay of nothing at all is exp(-10^4), which is zero too and leaves differences of sums finite
      float g = in ? a.log_decay[row] : 0.f;
      g = g < -1e4f ? -1e4f : g;
      const int start = in && a.starts ? a.starts[(int64_t)b * a.t + t] != 0 : 0;
      double sum = g;
      int n = start;
      for (int o = 1; o < 64; o <<= 1) {
        const int m = __shfl_up(n, o);
        if (lane >= o) n += m;
      }
      // within a sequence only: what is not finite must not reach the next one's differences
      for (int o = 1; o < 64; o <<= 1) {
        const double s = __shfl_up(sum, o);
        const int m = __shfl_up(n, o);
        if (lane >= o && m == n) sum += s;
      }
      const double all = __shfl(sum, 63);
      const int last = __shfl(n, 63);
      sums[lane] = sum;
      seq[lane] = n;
      beta[lane] = bt;
      float* rows = a.w.rows + at * 4 * kChunk;
      rows[lane] = n == 0 ? expf((float)sum) : 0.f;
      rows[kChunk + lane] = n == last ? expf((float)(all - sum)) : 0.f;
      rows[2 * kChunk + lane] = bt;
      rows[3 * kChunk + lane] = start ? 0.f : expf(g);
      if (backward) {
        a.w.sums[at * kChunk + lane] = sum;
        a.w.seq[at * kChunk + lane] = n;
      }
    }
    k.put(ks, a.dkp);
    q.put(qs, a.dkp);
  }
  __syncthreads();
  // wave w: rows 16 w .. + 15 of k k^T and q k^T
  {
    const int q4 = lane / 16, m = lane % 16;
    for (int tj = 0; tj < 4; ++tj) {
      f32x4_t kk = {0.f, 0.f, 0.f, 0.f}, qk = kk;
      if (tj <= wave)
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
          const int col = 32 * s + 8 * q4;
          const auto kb = natural<NP>(ks + (16 * tj + m) * RowsAt<DK>::stride + col, RowsAt<DK>::part);
          kk = mma(natural<NP>(ks + (16 * wave + m) * RowsAt<DK>::stride + col, RowsAt<DK>::part), kb, kk);
          qk = mma(natural<NP>(qs + (16 * wave + m) * RowsAt<DK>::stride + col, RowsAt<DK>::part), kb, qk);
        }
      const int j = 16 * tj + m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * wave + 4 * q4 + r;
        const bool same = j <= i && seq[i] == seq[j];
        const float d = same ? expf((float)(sums[i] - sums[j])) : 0.f;
        low[i * kLd + j] = same && j < i ? d * kk[r] : 0.f;
        read[i * kLd + j] = same ? d * qk[r] : 0.f;
      }
    }
  }
  __syncthreads();
  // column `lane` of H, row by row: h_i = -L_i - sum over k < i of L_ik beta_k h_k
  if (wave == 0) {
    float hc[kChunk], bh_[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      float acc = -low[i * kLd + lane];
#pragma unroll
      for (int k = 0; k < i; ++k) acc = fmaf(-low[i * kLd + k], bh_[k], acc);
      hc[i] = lane < i ? acc : 0.f;
      bh_[i] = lane < i ? beta[i] * acc : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i) low[i * kLd + lane] = hc[i];
  }
  __syncthreads();
  put_matrix<false>(low, a.w.solve + at * kMatrix);
  if (!backward) {
    put_matrix<false>(read, a.w.read + at * kMatrix);
  } else {
    put_matrix<true>(low, a.w.solve_t + at * kMatrix);
    put_matrix<true>(read, a.w.read_t + at * kMatrix);
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
  __builtin_memcpy(__builtin_assume_aligned((T*)a.w.q + i * 8, 16), vq, sizeof(vq));
  __builtin_memcpy(__builtin_assume_aligned((T*)a.w.k + i * 8, 16), vk, sizeof(vk));
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
