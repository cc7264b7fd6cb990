// norm_device.h -- device helpers shared by the group norm's kernels.
#pragma once

#include "norm_params.h"
#include "seq_device.h"

#pragma clang fp contract(off)

namespace convnorm {

using convseq::No;
using convseq::Pack;
using convseq::Yes;

__device__ __forceinline__ float param(const void* p, int f32, int dtype, int64_t at, float none) {
  if (!p) return none;
  if (f32) return ((const float*)p)[at];
  return dtype == convfwd::kF16 ? (float)((const _Float16*)p)[at] : (float)((const __bf16*)p)[at];
}

// 1 / (1 + e^-z): the hardware's exponential and reciprocal, an ulp each.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

// z * sigmoid(z) and, for the gradient, its derivative.
template <bool SILU>
__device__ __forceinline__ float activate(float z) {
  return SILU ? z * sigmoid(z) : z;
}
template <bool SILU>
__device__ __forceinline__ float slope(float z) {
  if (!SILU) return 1.f;
  const float s = sigmoid(z);
  return s * fmaf(z, 1.f - s, 1.f);
}

// Sum over the lanes of a team (a power of two of neighbouring lanes, at most a wave).
__device__ __forceinline__ float team_sum(float v, int team) {
  for (int o = 1; o < team; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

template <int N>
struct Int {
  static constexpr int value = N;
};

template <typename F>
inline hipError_t for_kind(int dtype, int v, int act, const F& f) {
  const auto act_of = [&](auto t, auto vec) {
    return act ? f(t, vec, Yes{}) : f(t, vec, No{});
  };
  if (dtype == convfwd::kF32) return v == 1 ? act_of(float{}, Int<1>{}) : act_of(float{}, Int<4>{});
  if (dtype == convfwd::kF16) return v == 1 ? act_of(_Float16{}, Int<1>{}) : act_of(_Float16{}, Int<8>{});
  return v == 1 ? act_of(__bf16{}, Int<1>{}) : act_of(__bf16{}, Int<8>{});
}

}  // namespace convnorm
