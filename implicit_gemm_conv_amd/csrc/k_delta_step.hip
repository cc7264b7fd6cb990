// k_delta_step.hip -- gated delta rule, one row of each of many streams: the state
// is read once, written once, and held in registers in between.  Bound by memory: 128
// streams of 16 heads of 128 x 128 move 268 MB in 47 us, 5.7 TB/s; one stream of 4 heads
// of 64 x 64 takes 4.1 us, most of it latency.
#include "delta_device.h"

namespace convdelta {

namespace {

// A workgroup owns 64 columns of one head of one stream; thread (dg, vc) holds the
// columns 4 vc .. + 3 of the rows d = dg + 16 n.
constexpr int kT = 256, kCols = 64, kHeld = kMaxDk / 16;

__device__ __forceinline__ f32x4_t load4(const float* p, int left, bool whole) {
  if (whole) return *(const f32x4_t*)p;
  f32x4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = e < left ? p[e] : 0.f;
  return v;
}

template <typename T>
__global__ __launch_bounds__(kT) void delta_step_kernel(DeltaStepArgs a, int blocks) {
  __shared__ float kq[2][kMaxDk];
  __shared__ f32x4_t part[kT / 64][16];
  const int cb = blockIdx.x % blocks, bh = blockIdx.x / blocks, b = bh / a.hv, h = bh % a.hv, hk = h / (a.hv / a.hk);
  const int vc = threadIdx.x % 16, dg = threadIdx.x / 16, col = cb * kCols + 4 * vc;
  const int slot = a.slots ? a.slots[b] : b, left = a.dv - col;
  T* y = (T*)a.y + (int64_t)bh * a.dv + col;
  if (slot < 0 || slot >= a.n_slots) {
    if (dg == 0)
      for (int e = 0; e < 4; ++e)
        if (e < left) y[e] = from_f32<T>(0.f);
    return;
  }
  const int64_t base = ((int64_t)slot * a.hv + h) * a.dk * a.dv + col;
  const bool whole = a.dv % 4 == 0 && left > 0 && ((uintptr_t)a.state | (uintptr_t)a.state_out) % 16 == 0;
  f32x4_t s[kHeld];
#pragma unroll
  for (int n = 0; n < kHeld; ++n) {
    const int d = dg + 16 * n;
    s[n] = d < a.dk ? load4(a.state + base + (int64_t)d * a.dv, left, whole) : f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  if ((int)threadIdx.x < kMaxDk) {
    const int d = threadIdx.x;
    kq[0][d] = d < a.dk ? to_f32(((const T*)a.k.p)[b * a.k.sb + hk * a.k.sh + d]) : 0.f;
    kq[1][d] = d < a.dk ? to_f32(((const T*)a.q.p)[b * a.q.sb + hk * a.q.sh + d]) : 0.f;
  }
  const float decay = expf(a.log_decay[bh]), beta = a.beta[bh];
  f32x4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = e < left ? to_f32(((const T*)a.v.p)[b * a.v.sb + h * a.v.sh + col + e]) : 0.f;
  __syncthreads();
  // the 16 row groups' parts, each four lanes' of a wave first, then the waves'
  const auto over_rows = [&](f32x4_t p) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] += __shfl_xor(p[e], 16);
      p[e] += __shfl_xor(p[e], 32);
    }
    if (threadIdx.x % 64 < 16) part[threadIdx.x / 64][vc] = p;
    __syncthreads();
    p = part[0][vc];
    for (int w = 1; w < kT / 64; ++w) p += part[w][vc];
    __syncthreads();
    return p;
  };
  f32x4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = 0; n < kHeld; ++n) {
    const float kd = kq[0][dg + 16 * n];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[n][e] = times(decay, s[n][e]);
      if (dg + 16 * n < a.dk) p[e] = fmaf(s[n][e], kd, p[e]);
    }
  }
  p = over_rows(p);
  f32x4_t u, o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = beta * (v[e] - p[e]);
#pragma unroll
  for (int n = 0; n < kHeld; ++n) {
    const int d = dg + 16 * n;
    if (d >= a.dk) continue;
    const float kd = kq[0][d], qd = kq[1][d];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[n][e] = fmaf(kd, u[e], s[n][e]);
      o[e] = fmaf(s[n][e], qd, o[e]);
    }
    float* to = a.state_out + base + (int64_t)d * a.dv;
    if (whole) {
      *(f32x4_t*)to = s[n];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) to[e] = s[n][e];
    }
  }
  o = over_rows(o);
  if (dg == 0)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) y[e] = from_f32<T>(a.scale * o[e]);
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s) {
  return for_type(a.dtype, [&](auto t) {
    const int blocks = (a.dv + kCols - 1) / kCols;
    hipLaunchKernelGGL((delta_step_kernel<decltype(t)>), dim3((unsigned)(a.b * a.hv * blocks)), dim3(kT), 0, s, a, blocks);
    return hipGetLastError();
  });
}

}  // namespace convdelta
