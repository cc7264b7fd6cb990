// k_seq_scan.hip -- gated linear recurrence along a sequence: forward,
// backward and the single-row step of serving.
//
//   r = sigmoid(gate_r), i = sigmoid(gate_i), u = decay * softplus(lam) * r, a = e^-u
//   h_t = a_t h_{t-1} + m_t v_t,  m = sqrt(1 - a^2),  v = i * x
//
// Backward, with g_t the whole gradient of h_t, g_t = dy_t + a_{t+1} g_{t+1}:
//   dx = g m i,   dgate_i = g m x i (1 - i)
//   e = g u (v a^2 / m - a h_{t-1}),   dgate_r = e (1 - r),
//   dlam = (sigmoid(lam) / softplus(lam)) sum e
// (dm/du = a^2 / m; u a^2 / m goes to zero with u).
#include "seq_device.h"

namespace convseq {

namespace {

// The value (b, t, ch) of an input that comes as it was or in 8 bits.
template <typename T>
__device__ __forceinline__ float value(const Rows& x, const Kept& k, int b, int t, int ch, int tt, int c) {
  if (!k.q) return to_f32(((const T*)x.p)[b * x.sb + (int64_t)t * x.st + ch]);
  const int groups = (tt + kGroup - 1) / kGroup;
  const int64_t at = ((int64_t)b * groups + t / kGroup) * c + ch;
  return (float)k.q[at * kGroup + t % kGroup] * group_scale(k.e[at]);
}

// One thread per channel of a sequence: piece after piece from the last, h
// forward through the piece, then the gradient back through it.
template <typename T>
__global__ __launch_bounds__(64) void seq_scan_bwd_kernel(ScanArgs a) {
  const int cb = (a.c + 63) / 64;
  const int ch = (int)(blockIdx.x % cb) * 64 + threadIdx.x, b = blockIdx.x / cb;
  if (ch >= a.c) return;
  const float rate = channel_rate(a.lam[ch], a.decay);
  const int64_t bc = (int64_t)b * a.c + ch;
  const int pieces = (a.t + kEvery - 1) / kEvery;
  const uint8_t* starts = a.starts ? a.starts + (int64_t)b * a.t : nullptr;
  float g = a.dh_last ? a.dh_last[bc] : 0.f, sum = 0.f;
  for (int p = pieces - 1; p >= 0; --p) {
    const int t0 = p * kEvery, t1 = min(a.t, t0 + kEvery);
    float before[kEvery];
    float h = a.states_in[((int64_t)b * pieces + p) * a.c + ch];
    for (int t = t0; t < t1; ++t) {
      const float x = value<T>(a.x, a.kept[0], b, t, ch, a.t, a.c);
      const Gate k = gates(value<T>(a.r, a.kept[1], b, t, ch, a.t, a.c), value<T>(a.i, a.kept[2], b, t, ch, a.t, a.c), rate);
      const float in = k.t * inv_sqrt(k.t) * (k.i * x);
      before[t - t0] = h;
      h = starts && starts[t] ? in : fmaf(k.a, h, in);
    }
    for (int t = t1 - 1; t >= t0; --t) {
      const float x = value<T>(a.x, a.kept[0], b, t, ch, a.t, a.c);
      const Gate k = gates(value<T>(a.r, a.kept[1], b, t, ch, a.t, a.c), value<T>(a.i, a.kept[2], b, t, ch, a.t, a.c), rate);
      const float rs = inv_sqrt(k.t), m = k.t * rs;
      g += to_f32(((const T*)a.dy.p)[b * a.dy.sb + (int64_t)t * a.dy.st + ch]);
      const bool first = starts && starts[t];
      float q = k.i * x * (k.a * k.a) * rs;
      if (!first) q = fmaf(-k.a, before[t - t0], q);
      const float e = g * k.u * q, dv = g * m;
      const int64_t at = ((int64_t)b * a.t + t) * a.c + ch;
      ((T*)a.dx)[at] = from_f32<T>(dv * k.i);
      ((T*)a.di)[at] = from_f32<T>(dv * x * (k.i * (1.f - k.i)));
      ((T*)a.dr)[at] = from_f32<T>(e * (1.f - k.r));
      sum += e;
      g = first ? 0.f : g * k.a;
    }
  }
  if (a.dh0) a.dh0[bc] = g;
  ((float*)a.work)[bc] = sum;
}

__global__ __launch_bounds__(64) void seq_scan_sum_kernel(const float* work, int parts, int c, const float* lam,
                                                          float* dlam) {
  const int ch = blockIdx.x * 64 + threadIdx.x;
  if (ch >= c) return;
  float s = 0.f;
  for (int p = 0; p < parts; ++p) s += work[(int64_t)p * c + ch];
  dlam[ch] = s * channel_unit(lam[ch]);
}

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
  const Gate g = gates(to_f32(((const T*)a.r)[b * a.r_row + ch]), to_f32(((const T*)a.i)[b * a.i_row + ch]),
                       channel_rate(a.lam[ch], a.decay));
  const float in = g.t * inv_sqrt(g.t) * (g.i * to_f32(((const T*)a.x)[b * a.x_row + ch]));
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

int64_t scan_bwd_work_bytes(int b, int, int c) { return (int64_t)b * c * 4; }

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s) {
  return for_type(a.dtype, [&](auto t) {
    if (a.b > 0)
      hipLaunchKernelGGL((seq_scan_bwd_kernel<decltype(t)>), dim3((a.c + 63) / 64 * a.b), dim3(64), 0, s, a);
    hipLaunchKernelGGL(seq_scan_sum_kernel, dim3((a.c + 63) / 64), dim3(64), 0, s, (const float*)a.work, a.b, a.c,
                       a.lam, a.dlam);
    return hipGetLastError();
  });
}

hipError_t launch_scan_step(const ScanStepArgs& a, hipStream_t s) {
  return for_type(a.dtype, [&](auto t) {
    hipLaunchKernelGGL((seq_scan_step_kernel<decltype(t)>), dim3((a.c + 255) / 256 * a.b), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace convseq
