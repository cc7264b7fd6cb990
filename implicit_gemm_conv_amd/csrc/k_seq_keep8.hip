// k_seq_keep8.hip -- a (B, T, C) tensor into 8 bits and back.  Groups of 16
// consecutive rows of one channel share a power of two: down a channel values
// are of one scale where channels of one row are not, and neighbouring lanes
// hold neighbouring channels, so the largest of a group needs no exchange
// between lanes.
#include "seq_device.h"

namespace convseq {

namespace {

// One thread per channel and group.
template <typename T>
__global__ __launch_bounds__(256) void pack8_kernel(int t, int c, int groups, Rows x, Kept k) {
  const int cb = (c + 255) / 256;
  const int ch = (int)(blockIdx.x % cb) * 256 + threadIdx.x, part = blockIdx.x / cb;
  if (ch >= c) return;
  const int b = part / groups, g = part % groups;
  const int t0 = g * kGroup, n = min(t - t0, kGroup);
  const T* p = (const T*)x.p + b * x.sb + (int64_t)t0 * x.st + ch;
  float v[kGroup];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    v[j] = j < n ? to_f32(p[(int64_t)j * x.st]) : 0.f;
    top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  const int byte = group_byte(top);
  const float inv = group_inverse(byte);
  k.e[(int64_t)part * c + ch] = (uint8_t)byte;
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < n) k.q[((int64_t)b * t + t0 + j) * c + ch] = (int8_t)quantise(v[j], inv);
}

template <typename T>
__global__ __launch_bounds__(256) void unpack8_kernel(int t, int c, int groups, Kept k, T* out) {
  const int cb = (c + 255) / 256;
  const int ch = (int)(blockIdx.x % cb) * 256 + threadIdx.x, part = blockIdx.x / cb;
  if (ch >= c) return;
  const int b = part / groups, g = part % groups;
  const int t0 = g * kGroup, n = min(t - t0, kGroup);
  const float scale = group_scale(k.e[(int64_t)part * c + ch]);
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < n) {
      const int64_t at = ((int64_t)b * t + t0 + j) * c + ch;
      out[at] = from_f32<T>((float)k.q[at] * scale);
    }
}

}  // namespace

hipError_t launch_pack8(int b, int t, int c, int dtype, const Rows& x, const Kept& k, hipStream_t s) {
  const int groups = (t + kGroup - 1) / kGroup;
  const dim3 grid((unsigned)((c + 255) / 256 * b * groups));
  if (dtype == convfwd::kF32)
    hipLaunchKernelGGL(pack8_kernel<float>, grid, dim3(256), 0, s, t, c, groups, x, k);
  else if (dtype == convfwd::kF16)
    hipLaunchKernelGGL(pack8_kernel<_Float16>, grid, dim3(256), 0, s, t, c, groups, x, k);
  else
    hipLaunchKernelGGL(pack8_kernel<__bf16>, grid, dim3(256), 0, s, t, c, groups, x, k);
  return hipGetLastError();
}

hipError_t launch_unpack8(int b, int t, int c, int dtype, const Kept& k, void* out, hipStream_t s) {
  const int groups = (t + kGroup - 1) / kGroup;
  const dim3 grid((unsigned)((c + 255) / 256 * b * groups));
  if (dtype == convfwd::kF32)
    hipLaunchKernelGGL(unpack8_kernel<float>, grid, dim3(256), 0, s, t, c, groups, k, (float*)out);
  else if (dtype == convfwd::kF16)
    hipLaunchKernelGGL(unpack8_kernel<_Float16>, grid, dim3(256), 0, s, t, c, groups, k, (_Float16*)out);
  else
    hipLaunchKernelGGL(unpack8_kernel<__bf16>, grid, dim3(256), 0, s, t, c, groups, k, (__bf16*)out);
  return hipGetLastError();
}

}  // namespace convseq
