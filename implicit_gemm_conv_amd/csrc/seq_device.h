// seq_device.h -- device helpers shared by the sequence kernels: the 8-bit
// format and the gates' mathematics.
#pragma once

#include "conv_device.h"
#include "seq_params.h"

// Every fused multiply-add is written as one; none is made from a product and a
// sum.  What the compiler fuses can differ between the variants of a kernel and
// between its code for whole and for ragged tiles, and a value would get
// different bits by where in a tile, or in how wide a lane, it is computed.
#pragma clang fp contract(off)

namespace convseq {

using convfwd::from_f32;
using convfwd::to_f32;

struct Yes {
  static constexpr bool value = true;
};
struct No {
  static constexpr bool value = false;
};

// The fp32 result itself, before it is rounded to T: the empty asm keeps the
// compiler from merging the last fp32 operation with the rounding to fp16 on
// some paths of a kernel and not on others, which would give a row different
// bits by where in a tile it lies.
template <typename T>
__device__ __forceinline__ T rounded(float f) {
  if (sizeof(T) == 2) asm("" : "+v"(f));
  return from_f32<T>(f);
}

// An access of 2 to 16 bytes as a plain type.
template <int N>
struct Words {
  typedef uint32_t type __attribute__((ext_vector_type(N / 4)));
};
template <>
struct Words<2> {
  typedef uint16_t type;
};
template <>
struct Words<4> {
  typedef uint32_t type;
};

// ---- V neighbouring channels of a row as one access ----
template <typename T, int V>
struct Pack;  // V * sizeof(T) bytes
template <typename T>
struct Pack<T, 1> {
  T v;
  __device__ __forceinline__ T word(int) const { return v; }
  __device__ __forceinline__ void put(int, T w) { v = w; }
  __device__ __forceinline__ float get(int) const { return to_f32(v); }
  __device__ __forceinline__ void set(int, float f) { v = rounded<T>(f); }
};
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  typedef T type __attribute__((ext_vector_type(V)));
  type v;
  __device__ __forceinline__ T word(int i) const { return v[i]; }
  __device__ __forceinline__ void put(int i, T w) { v[i] = w; }
  __device__ __forceinline__ float get(int i) const { return to_f32((T)v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = rounded<T>(f); }
};

// Makes the compiler take a held value as a new one: what was unpacked from it
// before is unpacked again where it is needed next, in one or two instructions,
// and not kept in registers in between.
template <typename P>
__device__ __forceinline__ void renew(P& p) {
  uint32_t w[(sizeof(P) + 3) / 4] = {};
  __builtin_memcpy(w, &p, sizeof(P));
#pragma unroll
  for (unsigned k = 0; k < sizeof(w) / 4; ++k) asm("" : "+v"(w[k]));
  __builtin_memcpy(&p, w, sizeof(P));
}

// An access at a wave-uniform base and a lane's byte offset of 32 bits, which the
// hardware adds itself: no 64-bit address a lane and row has to be computed and
// held.  The compiler sees that it may do so where the offset's widening stands in
// the same block of code: renew() the offset at the start of a block of accesses.
template <typename P>
__device__ __forceinline__ P load_at(const void* base, uint32_t offset) {
  return *(const P*)((const char*)base + offset);
}
template <typename P>
__device__ __forceinline__ void store_at(void* base, uint32_t offset, const P& v) {
  *(P*)((char*)base + offset) = v;
}

// Walks over rows `stride` bytes apart, one scalar addition a row.  The row's
// pointer is pinned to scalar registers: otherwise the compiler adds the lane's
// offset first and steps the sums, a 64-bit vector addition and a register pair a
// row.  (It is typed as global memory because the pinning hides where it came from.)
struct RowWalk {
  typedef __attribute__((address_space(1))) char* Global;
  Global at;
  int64_t stride;
  __device__ __forceinline__ RowWalk(const void* first, int64_t stride_) : at((Global)(uintptr_t)first), stride(stride_) {}
  // a step that is not taken repeats the row; one path for both, so that the loads
  // stay together where they are issued
  __device__ __forceinline__ void step(bool taken = true) { at += taken ? stride : 0; }
  template <typename P>
  __device__ __forceinline__ P load(uint32_t offset) {
    typedef typename Words<sizeof(P)>::type W;
    asm("" : "+s"(at));
    const W w = *(const __attribute__((address_space(1))) W*)(at + offset);
    P v;
    __builtin_memcpy(&v, &w, sizeof(P));
    return v;
  }
  template <typename P>
  __device__ __forceinline__ void store(uint32_t offset, const P& v) {
    typedef typename Words<sizeof(P)>::type W;
    asm("" : "+s"(at));
    W w;
    __builtin_memcpy(&w, &v, sizeof(P));
    *(__attribute__((address_space(1))) W*)(at + offset) = w;
  }
};

// ---- 8-bit groups ----
// Byte of a group whose largest magnitude has the float bits `top` (sign
// cleared; an unsigned maximum of the bits orders magnitudes and puts
// infinities and NaN on top).
__device__ __forceinline__ int group_byte(uint32_t top) {
  const int biased = (int)(top >> 23);
  return biased == 255 ? 255 : max(biased - 6, 1);
}
// 2^(127 - byte): what the group's values are multiplied by before rounding
// (for byte 255 it does not matter; such a group is read back as NaN).
__device__ __forceinline__ float group_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }
// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float group_scale(int byte) {
  return byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)byte << 23);
}
// The largest magnitudes' float bits of V channels over 16 rows.  16-bit types
// compare two channels at once in their own bits.
template <typename T, int V>
__device__ __forceinline__ void group_top(const Pack<T, V> (&raw)[kGroup], uint32_t (&top)[V]) {
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    typedef uint16_t pair __attribute__((ext_vector_type(2)));
    pair m[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) m[k] = (pair)(uint16_t)0;
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      uint32_t w[V / 2];
      __builtin_memcpy(w, &raw[j], sizeof(w));
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const uint32_t u = w[k] & 0x7fff7fffu;
        pair v;
        __builtin_memcpy(&v, &u, 4);
        m[k] = __builtin_elementwise_max(m[k], v);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      T t;
      const uint16_t bits = m[i / 2][i % 2];
      __builtin_memcpy(&t, &bits, 2);
      top[i] = __float_as_uint(to_f32(t));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      top[i] = 0;
#pragma unroll
      for (int j = 0; j < kGroup; ++j) top[i] = max(top[i], __float_as_uint(raw[j].get(i)) & 0x7fffffffu);
    }
  }
}
// Four values to four bytes, each rounded to nearest even within +-127: the
// scaling is exact (a power of two), and adding 1.5 * 2^23 leaves the rounded
// whole number in the low byte of the sum.
__device__ __forceinline__ uint32_t quantise4(float a, float b, float c, float d, float inverse) {
  constexpr float one = 12582912.f;
  const auto q = [&](float v) {
    return __float_as_uint(__builtin_amdgcn_fmed3f(fmaf(v, inverse, one), one - 127.f, one + 127.f));
  };
  // bytes 0 of two words side by side, twice
  const uint32_t lo = __builtin_amdgcn_perm(q(b), q(a), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(q(d), q(c), 0x0c0c0400u);
  return hi << 16 | lo;
}
// V channels from ch of group `at` (batch and group as one index) into 8 bits.
// raw: the group's rows, those past the first n (n >= 1) repeating one of them.
template <typename T, int V>
__device__ __forceinline__ void keep_group(const Pack<T, V> (&raw)[kGroup], int n, const Kept& k, int64_t at, int c,
                                           int ch) {
  uint32_t top[V];
  group_top<T, V>(raw, top);
  Pack<uint8_t, V> e;
  uint32_t w[4][V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int byte = group_byte(top[i]);
    const float inv = group_inverse(byte);
    e.put(i, (uint8_t)byte);
#pragma unroll
    for (int h = 0; h < 4; ++h)
      w[h][i] = quantise4(raw[4 * h].get(i), raw[4 * h + 1].get(i), raw[4 * h + 2].get(i), raw[4 * h + 3].get(i), inv);
    if (n < kGroup)
#pragma unroll
      for (int h = 0; h < 4; ++h) w[h][i] &= n >= 4 * h + 4 ? ~0u : n <= 4 * h ? 0u : (1u << 8 * (n - 4 * h)) - 1u;
  }
  store_at(k.e + at * c, (uint32_t)ch, e);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    Pack<uint32_t, 2 * V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      q.put(2 * i, w[2 * h][i]);
      q.put(2 * i + 1, w[2 * h + 1][i]);
    }
    store_at(k.q + (at * 2 + h) * c * 8, (uint32_t)ch * 8, q);
  }
}
// Rows 8 h .. 8 h + 7 of V channels: byte j % 4 of word j / 4 is row j.
template <int V>
struct Half {
  Pack<uint32_t, 2 * V> w;
  __device__ __forceinline__ float get(int i, int j) const {
    return (float)(int8_t)(w.word(2 * i + j / 4) >> 8 * (j % 4));
  }
};
template <int V>
__device__ __forceinline__ Half<V> half_group(const Kept& k, int64_t at, int h, int c, int ch) {
  return Half<V>{load_at<Pack<uint32_t, 2 * V>>(k.q + (at * 2 + h) * c * 8, (uint32_t)ch * 8)};
}
template <int V>
__device__ __forceinline__ void group_scales(const Kept& k, int64_t at, int c, int ch, float (&scale)[V]) {
  const Pack<uint8_t, V> e = load_at<Pack<uint8_t, V>>(k.e + at * c, (uint32_t)ch);
#pragma unroll
  for (int i = 0; i < V; ++i) scale[i] = group_scale(e.word(i));
}

// ---- gates ----
// The gates work in powers of two: exp2 and the reciprocals are the hardware's
// (1 ulp each), and log2 e is multiplied into what comes before them.
constexpr float kLog2e = 1.44269504f;

// 1 / (1 + 2^x), the sigmoid of -x ln 2: 1 and 0 at the infinities, NaN for NaN.
__device__ __forceinline__ float sigmoid2(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x));
}
__device__ __forceinline__ float sigmoid(float x) { return sigmoid2(-kLog2e * x); }

// softplus(l) = ln(1 + e^l) = max(l, 0) + 2 atanh(z), z = e / (2 + e), e = e^-|l|:
// z <= 1/3, the series to z^15 leaves less than 1e-8 of the sum, and a small
// softplus keeps its relative accuracy, which the decay rates near 0 need.
__device__ __forceinline__ float softplus(float l) {
  const float e = expf(-fabsf(l));
  const float z = e * __builtin_amdgcn_rcpf(2.f + e), s = z * z;
  float p = fmaf(s, 1.f / 15.f, 1.f / 13.f);
  p = fmaf(s, p, 1.f / 11.f);
  p = fmaf(s, p, 1.f / 9.f);
  p = fmaf(s, p, 1.f / 7.f);
  p = fmaf(s, p, 1.f / 5.f);
  p = fmaf(s, p, 1.f / 3.f);
  return fmaxf(l, 0.f) + 2.f * fmaf(s * z, p, z);
}
// d ln(softplus) / d lam = sigmoid(lam) / softplus(lam), 1 where both vanish.
__device__ __forceinline__ float channel_unit(float lam) {
  return lam < -80.f ? 1.f : 1.f / ((1.f + expf(-lam)) * softplus(lam));
}

// What multiplies the open gate r: u = rate r with rate = decay * softplus(lam), and
// log2 a = -rate log2 e r.
struct Rate {
  float u, log2;
};
__device__ __forceinline__ Rate rate_of(float u) { return Rate{u, -kLog2e * u}; }

// 1 - e^(-2u) for u >= 0, given a = e^-u.  Below u = 1/8, where 1 - a^2 would lose
// the leading bits, u times the polynomial of degree 4 nearest to (1 - e^(-2u)) / u
// there in relative error (at most 7e-9 off, fitted at Chebyshev points).
__device__ __forceinline__ float one_minus_square(float u, float a) {
  float p = fmaf(u, 0.2403048575f, -0.6638176441f);
  p = fmaf(u, p, 1.333206058f);
  p = fmaf(u, p, -1.999997973f);
  p = fmaf(u, p, 2.f);
  return u < 0.125f ? u * p : fmaf(-a, a, 1.f);
}

// a and its products are positive numbers, and are kept so where fp32 would round
// them to zero (to 2^-149, its smallest number): an infinite state stays infinite
// instead of becoming NaN, and every reader of a product computes with the same
// one.  A sign bit, and a NaN, stay as they are.
__device__ __forceinline__ float positive(float a) { return __uint_as_float(max(__float_as_uint(a), 1u)); }

// The gates of one value; x2 are the logits times -log2 e.
struct Gate {
  float r, i, a, t;  // a = e^-u, t = 1 - a^2
};
__device__ __forceinline__ Gate gates(float r2, float i2, const Rate& rate) {
  Gate g;
  g.r = sigmoid2(r2);
  g.i = sigmoid2(i2);
  g.a = positive(__builtin_amdgcn_exp2f(rate.log2 * g.r));
  g.t = one_minus_square(rate.u * g.r, g.a);
  return g;
}
// t^(-1/2).  Where t vanishes it stays finite, so that products with t and u take
// their limit 0; a NaN in t is not passed on, but stays in t.
__device__ __forceinline__ float inv_sqrt(float t) { return __builtin_amdgcn_rsqf(fmaxf(t, 1e-36f)); }

// A barrier for what went through LDS alone: unlike __syncthreads it does not
// wait for global loads in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace convseq
