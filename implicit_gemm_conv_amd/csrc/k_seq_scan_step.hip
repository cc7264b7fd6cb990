// k_seq_scan_step.hip -- gated linear recurrence, one row of each of many
// streams: one lane a channel, bound by the launch (1 stream of 256 channels 1.8 us,
// 256 streams of 2048 4.1 us).
#include "seq_device.h"

namespace convseq {

namespace {

template <typename T>
__global__ __launch_bounds__(256) void seq_scan_step_kernel(ScanStepArgs a) {
  const int cb = (a.c + 255) / 256;
  const int ch = (int)(blockIdx.x % cb) * 256 + threadIdx.x, b = blockIdx.x / cb;
  if (ch >= a.c) return;
  T* y = (T*)a.y + (int64_t)b * a.c + ch;
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {
    *y = from_f32<T>(0.f);
    return;
  }
  const Gate g = gates(-kLog2e * to_f32(((const T*)a.r)[b * a.r_row + ch]),
                       -kLog2e * to_f32(((const T*)a.i)[b * a.i_row + ch]), rate_of(a.decay * softplus(a.lam[ch])));
  const float in = __builtin_amdgcn_sqrtf(g.t) * (g.i * to_f32(((const T*)a.x)[b * a.x_row + ch]));
  const float h = fmaf(g.a, a.state[(int64_t)slot * a.c + ch], in);
  a.state_out[(int64_t)slot * a.c + ch] = h;
  *y = from_f32<T>(h);
}

template <typename F>
hipError_t for_type(int dtype, const F& f) {
  if (dtype == convfwd::kF32) return f(float{});
  if (dtype == convfwd::kF16) return f(_Float16{});
  return f(__bf16{});
}

}  // namespace

hipError_t launch_scan_step(const ScanStepArgs& a, hipStream_t s) {
  return for_type(a.dtype, [&](auto t) {
    hipLaunchKernelGGL((seq_scan_step_kernel<decltype(t)>), dim3((a.c + 255) / 256 * a.b), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace convseq
