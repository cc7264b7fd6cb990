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

// What a channel's rate = decay * softplus(lam) multiplies the open gate by.
struct Rate {
  float u;     // u = rate * r
  float log2;  // log2 a = -rate log2 e * r
};
__device__ __forceinline__ Rate channel_rate(float lam, float decay) {
  const float u = decay * softplus(lam);
  return Rate{u, -kLog2e * u};
}

// 1 - e^(-2u) for u >= 0, given a = e^-u.  Below 2u = 1/4 by its series to (2u)^6
// (the next term is under 5e-8 of the sum), where 1 - a^2 would lose the leading bits.
__device__ __forceinline__ float one_minus_square(float u, float a) {
  float p = fmaf(u, -64.f / 720.f, 32.f / 120.f);
  p = fmaf(u, p, -16.f / 24.f);
  p = fmaf(u, p, 8.f / 6.f);
  p = fmaf(u, p, -2.f);
  p = fmaf(u, p, 2.f);
  return u < 0.125f ? u * p : fmaf(-a, a, 1.f);
}

// The gates of one value; x2 are the logits times -log2 e.
struct Gate {
  float r, i, a;  // a = e^-u
  float t, rs;    // 1 - a^2 and its inverse square root, so that m = t rs.  Where t vanishes rs stays
                  // finite, and products with m and u take their limit 0.  NaN stays NaN in t.
};
__device__ __forceinline__ Gate gates(float r2, float i2, const Rate& rate) {
  Gate g;
  g.r = sigmoid2(r2);
  g.i = sigmoid2(i2);
  g.a = __builtin_amdgcn_exp2f(rate.log2 * g.r);
  g.t = one_minus_square(rate.u * g.r, g.a);
  g.rs = __builtin_amdgcn_rsqf(fmaxf(g.t, 1e-36f));
  return g;
}

}  // namespace convseq
