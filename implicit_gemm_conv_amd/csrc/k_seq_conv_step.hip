// k_seq_conv_step.hip -- causal depthwise convolution, one row of each of many
// streams: one lane a channel, bound by the launch (8 streams of 1024 channels,
// 4 taps: 2.6 us).
#include "seq_conv.h"

namespace convseq {

namespace {

template <typename T, int K>
__global__ __launch_bounds__(256) void seq_conv_step_kernel(ConvStepArgs a) {
  const int cb = (a.c + 255) / 256;
  const int ch = (int)(blockIdx.x % cb) * 256 + threadIdx.x, b = blockIdx.x / cb;
  if (ch >= a.c) return;
  T* y = (T*)a.y + (int64_t)b * a.c + ch;
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {
    *y = from_f32<T>(0.f);
    return;
  }
  const T* in = (const T*)a.state + (int64_t)slot * (K - 1) * a.c + ch;
  T* out = (T*)a.state_out + (int64_t)slot * (K - 1) * a.c + ch;
  T win[K];
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) win[k] = in[(int64_t)k * a.c];
  win[K - 1] = ((const T*)a.x)[b * a.x_row + ch];
  float z = a.bias ? to_f32(((const T*)a.bias)[ch]) : 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) z = fmaf(to_f32(((const T*)a.w)[(int64_t)ch * K + k]), to_f32(win[k]), z);
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) out[(int64_t)k * a.c] = win[k + 1];
  *y = from_f32<T>(a.act ? silu(z) : z);
}

template <typename T>
hipError_t run(const ConvStepArgs& a, hipStream_t s) {
  return for_taps(a.k, [&](auto k) {
    hipLaunchKernelGGL((seq_conv_step_kernel<T, decltype(k)::value>), dim3((a.c + 255) / 256 * a.b), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t s) {
  if (a.dtype == convfwd::kF32) return run<float>(a, s);
  if (a.dtype == convfwd::kF16) return run<_Float16>(a, s);
  return run<__bf16>(a, s);
}

}  // namespace convseq
