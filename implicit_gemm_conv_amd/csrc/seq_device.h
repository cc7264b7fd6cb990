// seq_device.h -- device helpers shared by the sequence kernels: the 8-bit
// format and the gates' mathematics.
#pragma once

#include "conv_device.h"
#include "seq_params.h"

namespace convseq {

using convfwd::from_f32;
using convfwd::to_f32;

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
