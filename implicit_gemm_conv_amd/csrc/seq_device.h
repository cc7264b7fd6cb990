// seq_device.h -- device helpers shared by the sequence kernels: the 8-bit
// format and the gates' mathematics.
#pragma once

#include "conv_device.h"
#include "seq_params.h"

namespace convseq {

using convfwd::from_f32;
using convfwd::to_f32;

struct Yes {
  static constexpr bool value = true;
};
struct No {
  static constexpr bool value = false;
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
// (byte 255 gives 0; such a group is read back as NaN whatever it holds).
__device__ __forceinline__ float group_inverse(int byte) {
  return byte == 255 ? 0.f : __uint_as_float((uint32_t)(254 - byte) << 23);
}
// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float group_scale(int byte) {
  return byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)byte << 23);
}
// Round to nearest even within +-127.  The scaling is exact (a power of two;
// values it takes below the normal range round to zero either way).
__device__ __forceinline__ int quantise(float v, float inverse) {
  return (int)__builtin_rintf(__builtin_amdgcn_fmed3f(v * inverse, -127.f, 127.f));
}

// The 16 values of a group, of which n lie inside T, as 16 bytes; *byte gets
// the group's byte.
__device__ __forceinline__ uint4 pack_group(const float (&v)[kGroup], int n, int* byte) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < n) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  *byte = group_byte(top);
  const float inv = group_inverse(*byte);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * k + j < n) w[k] |= (uint32_t)(quantise(v[4 * k + j], inv) & 0xff) << (8 * j);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Byte j of four packed ones, as a signed number.
__device__ __forceinline__ float held(uint32_t w, int j) { return (float)(int8_t)(w >> (8 * j)); }

// The fp32 result itself, before it is rounded to T: the empty asm keeps the
// compiler from merging the last fp32 operation with the rounding to fp16 on
// some paths of a kernel and not on others, which would give a row different
// bits by where in a tile it lies.
template <typename T>
__device__ __forceinline__ T rounded(float f) {
  if (sizeof(T) == 2) asm("" : "+v"(f));
  return from_f32<T>(f);
}

// ---- V neighbouring channels of a row as one access ----
template <typename T, int V>
struct Pack;  // V * sizeof(T) bytes
template <typename T>
struct Pack<T, 1> {
  T v;
  __device__ __forceinline__ float get(int) const { return to_f32(v); }
  __device__ __forceinline__ void set(int, float f) { v = rounded<T>(f); }
};
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  typedef T type __attribute__((ext_vector_type(V)));
  type v;
  __device__ __forceinline__ float get(int i) const { return to_f32((T)v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = rounded<T>(f); }
};

// ---- gates ----
// 1 / (1 + 2^(-x log2 e)) on the hardware's exp2 and reciprocal (1 ulp each):
// 0 and 1 at the infinities, NaN for NaN.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}

// decay * softplus(lam), and d ln(softplus) / d lam = sigmoid(lam) / softplus(lam)
// (1 where both vanish).
__device__ __forceinline__ float channel_rate(float lam, float decay) {
  return decay * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam))));
}
__device__ __forceinline__ float channel_unit(float lam) {
  const float sp = fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam)));
  return lam < -80.f ? 1.f : 1.f / ((1.f + expf(-lam)) * sp);
}

// 1 - e^(-x) for x >= 0.  Below 1/4 by its series to x^6 (the next term is
// under 5e-8 of the sum), where 1 - e would lose the leading bits; above, from e = e^(-x).
__device__ __forceinline__ float one_minus_exp(float x, float e) {
  float p = fmaf(x, -1.f / 720.f, 1.f / 120.f);
  p = fmaf(x, p, -1.f / 24.f);
  p = fmaf(x, p, 1.f / 6.f);
  p = fmaf(x, p, -0.5f);
  p = fmaf(x, p, 1.f);
  return x < 0.25f ? x * p : 1.f - e;
}

// The gates of one value: u = rate * r, a = e^-u, t = 1 - a^2.
struct Gate {
  float r, i, u, a, t;
};
__device__ __forceinline__ Gate gates(float gr, float gi, float rate) {
  Gate g;
  g.r = sigmoid(gr);
  g.i = sigmoid(gi);
  g.u = rate * g.r;
  g.a = __builtin_amdgcn_exp2f(-1.44269504f * g.u);
  g.t = one_minus_exp(2.f * g.u, g.a * g.a);
  return g;
}
// 1 / sqrt(t); 0 where t vanishes, so that products with sqrt(t)'s factors
// take their limit 0 there.  NaN stays NaN.
__device__ __forceinline__ float inv_sqrt(float t) {
  return t < 1e-37f ? 0.f : __builtin_amdgcn_rsqf(t);
}

}  // namespace convseq
