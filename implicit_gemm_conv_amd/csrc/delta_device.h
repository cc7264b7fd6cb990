// delta_device.h -- device helpers shared by the gated delta rule's kernels.
//
// Mathematics of a chunk of 64 rows, with S the state before it.  G_i are the sums
// of log decays up to row i, D_ij = exp(G_i - G_j) for j <= i in the same sequence,
// L = D * (k k^T) below the diagonal and H = -(I + L beta)^-1 L, which is strictly
// lower triangular too.  Then
//
//   r = v - enter * (k S),  x = r + H (beta r),  u = beta x
//   y = scale * (enter * (q S) + R u),  R = D * (q k^T)
//   S <- enter_last * S + k^T (leave * u)
//
// where enter_i = exp(G_i) (zero from a start on) and leave_j = exp(G_last - G_j)
// (zero before the last start).  H holds no beta, so a beta of zero is nothing special.
//
// Products run on the bf16 matrix units at fp32's precision: an fp32 value is the
// sum of three bf16 parts (8 significant bits each), and of the parts' products
// those that matter to 24 bits are added in fp32.  A bf16 input is one part, an
// fp16 input two.  bf16 has fp32's range but not its last value's neighbourhood: from 2^128 - 2^119
// on the first part rounds to infinity and the value counts as one (as NaN, with what is left of it).  At the other
// end the third part runs out of bf16's range first: from about 2^-95 down bits are lost, at 2^-110 the last.
//
// A workgroup of eight waves carries 16 or 32 columns of one head's state (or of its
// gradient), four of them in each of two roles.  Wave w of a role computes rows 16 w
// .. + 15 of a chunk's r, x and y, and each wave 16 rows of the state; the parts of what
// one step makes and the next one contracts over go through LDS, column by column, so
// that an operand is one 16-byte read.
#pragma once

#include "conv_device.h"
#include "delta_params.h"

#pragma clang fp contract(off)

namespace convdelta {

using convfwd::bf168_t;
using convfwd::f32x4_t;
using convfwd::from_f32;
using convfwd::to_f32;

typedef __bf16 bf164_t __attribute__((ext_vector_type(4)));

// The wave's number in its workgroup, known to be one for all lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// The six (16-row tile, step of 32) pairs that hold something of a strictly or non-strictly
// lower triangle, and of its transpose.
__device__ constexpr int low_t(int f) { return f < 2 ? f : f < 4 ? 2 : 3; }
__device__ constexpr int low_s(int f) { return f < 2 ? 0 : f & 1; }
__device__ constexpr int up_t(int f) { return f < 4 ? f >> 1 : f - 2; }
__device__ constexpr int up_s(int f) { return f < 4 ? f & 1 : 1; }

// Parts of an input of type T.
template <typename T> struct InParts;
template <> struct InParts<__bf16> { static constexpr int n = 1; };
template <> struct InParts<_Float16> { static constexpr int n = 2; };
template <> struct InParts<float> { static constexpr int n = 3; };

template <int N>
struct Parts {
  bf168_t p[N];
};

template <int N>
__device__ __forceinline__ void split_one(float x, __bf16 (&o)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    o[k] = (__bf16)x;
    x -= (float)o[k];
  }
}

template <int N>
__device__ __forceinline__ Parts<N> split(const float (&x)[8]) {
  Parts<N> r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    __bf16 o[N];
    split_one<N>(x[e], o);
#pragma unroll
    for (int k = 0; k < N; ++k) r.p[k][e] = o[k];
  }
  return r;
}

// acc += A B from parts, the products that matter to fp32.
template <int NA, int NB>
__device__ __forceinline__ f32x4_t mma(const Parts<NA>& a, const Parts<NB>& b, f32x4_t acc) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < kParts) acc = convfwd::mfma16x16x32(a.p[i], b.p[j], acc);
  return acc;
}

// What is not wanted is selected away, not multiplied by zero.
__device__ __forceinline__ float times(float factor, float x) { return factor == 0.f ? 0.f : factor * x; }
__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// ---- rows of q, k in LDS: [part][64][DK + 8] bf16 ----
// The 8 spare elements spread the rows over the banks.
template <int DK>
struct RowsAt {
  static constexpr int stride = DK + 8, part = kChunk * stride;
};

// An access at a wave-uniform base and a lane's byte offset of 32 bits, which the hardware adds itself.
template <typename P>
__device__ __forceinline__ P load_at(const void* base, uint32_t offset) {
  return *(const P*)((const char*)base + offset);
}

// Accesses whose range the hardware checks: what lies past `bytes` is read as zero and not written.  No
// access needs a branch then, and the compiler knows how many are in flight at every wait (it counts them in the
// order of issue, and would take each that a branch may skip for one that was).
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every range
struct Range {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Range(const void* base, int64_t bytes)
      : r(__builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)bytes, 0x00027000)) {}
  template <typename T>
  __device__ __forceinline__ T load(uint32_t offset) const {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, offset, 0, 0));
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, offset, 0, 0));
    if constexpr (sizeof(T) == 8) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b64(r, offset, 0, 0));
    if constexpr (sizeof(T) == 16) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0));
  }
  template <typename T>
  __device__ __forceinline__ void store(uint32_t offset, T v) const {
    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, v), r, offset, 0, 0);
    if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned int, v), r, offset, 0, 0);
  }
};
// At the end of a path that is hardly ever taken: with nothing of it in flight, the waits after it are those of the
// usual path.
__device__ __forceinline__ void wait_for_memory() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

// The rows [t0, t) of one head, at most 64, of d elements.
template <typename T>
__device__ __forceinline__ Range rows_range(const Heads& h, int b, int head, int t0, int t, int d) {
  return Range((const T*)h.p + b * h.sb + head * h.sh + t0 * h.st, ((int64_t)(min(kChunk, t - t0) - 1) * h.st + d) * (int64_t)sizeof(T));
}
template <typename T>
__device__ __forceinline__ uint32_t row_bytes(const Heads& h) {
  return (uint32_t)h.st * (uint32_t)sizeof(T);
}

// 8 elements of a row as they come from memory; they stay raw until they are used, so
// that a load in flight is not waited for.  The row is 16-byte aligned and has d elements, a
// multiple of 8; past its end they are zero.
template <typename T>
struct Raw8 {
  convfwd::u32x4_t w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const Range& x, uint32_t row, int d0, int d) {
    const uint32_t at = d0 < d ? row + (uint32_t)d0 * (uint32_t)sizeof(T) : kNowhere;
#pragma unroll
    for (unsigned k = 0; k < sizeof(T) / 2; ++k) w[k] = x.load<convfwd::u32x4_t>(at + 16 * k);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    T v[8];
    __builtin_memcpy(v, w, sizeof(v));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = to_f32(v[e]);
  }
  __device__ __forceinline__ Parts<InParts<T>::n> parts() const {
    float x[8];
    get(x);
    return split<InParts<T>::n>(x);
  }
};
template <>
__device__ __forceinline__ Parts<1> Raw8<__bf16>::parts() const {
  Parts<1> r;
  __builtin_memcpy(&r.p[0], w, 16);
  return r;
}

// Pieces of a chunk's rows that a thread of `threads` holds on their way to LDS.
template <typename T, int DK, int THREADS>
struct Rows64 {
  static constexpr int pieces = kChunk * (DK / 8), each = (pieces + THREADS - 1) / THREADS;
  Raw8<T> p[each];
  __device__ __forceinline__ static int at(int k) { return min((int)threadIdx.x + k * THREADS, pieces - 1); }
  __device__ __forceinline__ static int row(int k) { return at(k) / (DK / 8); }
  __device__ __forceinline__ static int d0(int k) { return at(k) % (DK / 8) * 8; }
  __device__ __forceinline__ void load(const Heads& h, int b, int head, int t0, int t, int d) {
    const Range x = rows_range<T>(h, b, head, t0, t, d);
#pragma unroll
    for (int k = 0; k < each; ++k) p[k].load(x, row(k) * row_bytes<T>(h), d0(k), d);
  }
  __device__ __forceinline__ bool finite() const {
    bool all = true;
#pragma unroll
    for (int k = 0; k < each; ++k) {
      float x[8];
      p[k].get(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) all = all && convdelta::finite(x[e]);
    }
    return all;
  }
  __device__ __forceinline__ void put(__bf16* lds) const {
#pragma unroll
    for (int k = 0; k < each; ++k) {
      const auto q = p[k].parts();
#pragma unroll
      for (int n = 0; n < InParts<T>::n; ++n)
        *(bf168_t*)(lds + n * RowsAt<DK>::part + row(k) * RowsAt<DK>::stride + d0(k)) = q.p[n];
    }
  }
};

// 8 neighbouring elements of a row (or column) of parts in LDS: an operand.
template <int N>
__device__ __forceinline__ Parts<N> natural(const __bf16* at, int part) {
  Parts<N> r;
#pragma unroll
  for (int n = 0; n < N; ++n) r.p[n] = *(const bf168_t*)(at + n * part);
  return r;
}

// The transposed read: of 8 neighbouring rows of 16-bit values, row0 .. row0 + 7 for the lane's
// quarter, this lane's column.  The hardware reads 4 rows x 16 columns a quarter of the wave, each
// lane 4 neighbouring columns; lane p of a quarter points at row p / 4, and at the columns that the
// lanes 4 (p % 4) .. + 3 get.  `at` is that address for the first four rows.
template <int N>
__device__ __forceinline__ Parts<N> transposed(const __bf16* at, int stride, int part) {
  typedef __attribute__((address_space(3))) bf164_t* Lds;
  Parts<N> r;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const bf164_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Lds)(at + n * part));
    const bf164_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Lds)(at + n * part + 4 * stride));
    r.p[n] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  return r;
}

// Keeps the elements whose index k0 + e lies in [lo, hi).
template <int N>
__device__ __forceinline__ void keep(Parts<N>& a, int k0, int lo, int hi) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k0 + e < lo || k0 + e >= hi) a.p[n][e] = (__bf16)0.f;
}

__device__ __forceinline__ int64_t chunk_index(const DeltaArgs& a, int bh, int c) { return (int64_t)bh * a.chunks + c; }

// Workgroups of one head lie on one die (ids are dealt round-robin to 8), so that they share its L2.
__device__ __forceinline__ bool head_of(int heads, int blocks, int& bh, int& cb) {
  const int slot = blockIdx.x / 8;
  bh = slot / blocks * 8 + blockIdx.x % 8;
  cb = slot % blocks;
  return bh < heads;
}

template <typename F>
inline hipError_t for_type(int dtype, const F& f) {
  if (dtype == convfwd::kF32) return f(float{});
  if (dtype == convfwd::kF16) return f(_Float16{});
  return f(__bf16{});
}
template <int N>
struct Int {
  static constexpr int value = N;
};
// Head sizes are padded to 32, 64 or 128 inside the kernels (4x4096 rows, 16 heads of Dk x 128, bf16, forward and backward:
// Dk = 64 takes 298 and 635 us, padded to 128 320 and 752; Dk = 32 278 and 563, padded 303 and 714).
template <typename F>
inline hipError_t for_dk(int dk, const F& f) {
  if (dk <= 32) return f(Int<32>{});
  if (dk <= 64) return f(Int<64>{});
  return f(Int<128>{});
}

// The recurrences' columns a workgroup, in tiles of 16: one where the workgroups are then no more than the 256 CUs (two
// would leave more of them idle), and two, which read q, k and the chunks' matrices once for both, where they are more.
// 4096 rows of 128 x 128, states kept, one tile and two, forward and backward pass as called:
//   16 heads, bf16 (128 workgroups of one tile)   181 and 308 us, 255 and 371
//   32 heads, bf16 (256)                          231 and 474,    279 and 530
//   36 heads, bf16 (288)                          415 and 677,    302 and 575
//   64 heads, bf16 (512)                          511 and 955,    368 and 836
//   32 and 36 heads, fp32, forward alone          343 and 611,    411 and 433
// and with heads of 64 x 64 the same way (64 heads 254 and 281 us forward, 80 heads 441 and 320).
template <typename F>
inline hipError_t for_columns(const DeltaArgs& a, const F& f) {
  return (int64_t)a.b * a.hv * ((a.dv + 15) / 16) > 256 ? f(Int<2>{}) : f(Int<1>{});
}

}  // namespace convdelta
