// k_seq_conv.hip -- causal depthwise convolution along a sequence: forward,
// backward and the single-row step of serving.
//
//   z_t = bias + sum_k w_k X(t - (K-1) + k),   y = z or z * sigmoid(z)
//
// X is x, below row 0 the carried rows, and zero across a start.  How far back
// row t may look, reach(t) = min(K-1, t - (last start <= t)), depends on (b, t)
// alone, so it is the same for every lane of a wave: a tap j rows back counts
// iff j <= reach(t), and is selected, not multiplied, away.
#include "seq_device.h"

namespace convseq {

namespace {

constexpr int kPiece = 64;  // rows of a backward piece

__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }
__device__ __forceinline__ float silu_grad(float z) {
  const float s = sigmoid(z);
  return s * fmaf(z, 1.f - s, 1.f);
}

// reach(t - 1) for the row before t (rows before row 0 reach everything).
__device__ __forceinline__ int reach_before(const uint8_t* starts, int t, int k) {
  if (!starts) return k - 1;
  for (int j = 1; j < k && t - j >= 0; ++j)
    if (starts[t - j]) return j - 1;
  return k - 1;
}

template <typename T>
__device__ __forceinline__ float row_before(const T* x, int64_t st, const T* state, int s, int k, int c) {
  // X at s < 0: carried row s + K-1 of the batch's state
  return s >= 0 ? to_f32(x[(int64_t)s * st]) : state ? to_f32(state[(int64_t)(s + k - 1) * c]) : 0.f;
}

// One thread per channel and group of 16 rows.
template <typename T, int K>
__global__ __launch_bounds__(256) void seq_conv_fwd_kernel(ConvArgs a) {
  const int cb = (a.c + 255) / 256;
  const int ch = (int)(blockIdx.x % cb) * 256 + threadIdx.x, part = blockIdx.x / cb;
  if (ch >= a.c) return;
  const int groups = max(1, (a.t + kGroup - 1) / kGroup);
  const int b = part / groups, g = part % groups;
  const int t0 = g * kGroup, t1 = min(a.t, t0 + kGroup);
  const T* x = (const T*)a.x.p + b * a.x.sb + ch;
  const T* state = a.state ? (const T*)a.state + (int64_t)b * (K - 1) * a.c + ch : nullptr;
  const uint8_t* starts = a.starts ? a.starts + (int64_t)b * a.t : nullptr;
  T* y = (T*)a.y + (int64_t)b * a.t * a.c + ch;
  float w[K], win[K];
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = to_f32(((const T*)a.w)[(int64_t)ch * K + k]);
  const float bias = a.bias ? to_f32(((const T*)a.bias)[ch]) : 0.f;
#pragma unroll
  for (int k = 1; k < K; ++k) win[k] = row_before(x, a.x.st, state, t0 - K + k, K, a.c);
  int reach = reach_before(starts, t0, K);
  uint32_t top = 0;
  for (int t = t0; t < t1; ++t) {
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) win[k] = win[k + 1];
    win[K - 1] = to_f32(x[(int64_t)t * a.x.st]);
    top = max(top, __float_as_uint(win[K - 1]) & 0x7fffffffu);
    reach = starts && starts[t] ? 0 : min(reach + 1, K - 1);
    float z = bias;
#pragma unroll
    for (int k = 0; k < K; ++k) z = K - 1 - k <= reach ? fmaf(w[k], win[k], z) : z;
    y[(int64_t)t * a.c] = from_f32<T>(a.act ? silu(z) : z);
  }
  if (a.kept.q && t0 < t1) {
    const int byte = group_byte(top);
    const float inv = group_inverse(byte);
    a.kept.e[((int64_t)b * groups + g) * a.c + ch] = (uint8_t)byte;
    int8_t* q = a.kept.q + (((int64_t)b * groups + g) * a.c + ch) * kGroup;
    for (int j = 0; j < kGroup; ++j)
      q[j] = t0 + j < t1 ? (int8_t)quantise(to_f32(x[(int64_t)(t0 + j) * a.x.st]), inv) : 0;
  }
  if (a.state_out && g == groups - 1) {
    T* out = (T*)a.state_out + (int64_t)b * (K - 1) * a.c + ch;
    reach = reach_before(starts, a.t, K);
    for (int j = 0; j < K - 1; ++j) {
      const int s = a.t - (K - 1) + j;
      const float v = row_before(x, a.x.st, state, s, K, a.c);
      out[(int64_t)j * a.c] = from_f32<T>(a.t - 1 - s <= reach || a.t == 0 ? v : 0.f);
    }
  }
}

// One thread per channel and piece of 64 rows: dz row by row, spread over the
// rows it came from; the piece also walks the K-1 rows after it, for what they
// send back.
template <typename T, int K>
__global__ __launch_bounds__(256) void seq_conv_bwd_kernel(ConvArgs a) {
  const int cb = (a.c + 255) / 256;
  const int ch = (int)(blockIdx.x % cb) * 256 + threadIdx.x, part = blockIdx.x / cb;
  if (ch >= a.c) return;
  const int pieces = max(1, (a.t + kPiece - 1) / kPiece);
  const int b = part / pieces, p = part % pieces;
  const int t0 = p * kPiece, t1 = min(a.t, t0 + kPiece), end = min(a.t, t1 + K - 1);
  const int groups = (a.t + kGroup - 1) / kGroup;
  const T* x = (const T*)a.x.p + b * a.x.sb + ch;
  const T* dy = (const T*)a.dy.p + b * a.dy.sb + ch;
  const T* state = a.state ? (const T*)a.state + (int64_t)b * (K - 1) * a.c + ch : nullptr;
  const uint8_t* starts = a.starts ? a.starts + (int64_t)b * a.t : nullptr;
  const auto row = [&](int s) -> float {
    if (s < 0 || !a.kept.q) return row_before(x, a.x.st, state, s, K, a.c);
    const int64_t at = ((int64_t)b * groups + s / kGroup) * a.c + ch;
    return (float)a.kept.q[at * kGroup + s % kGroup] * group_scale(a.kept.e[at]);
  };
  float w[K], win[K], acc[K], dw[K], db = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    w[k] = to_f32(((const T*)a.w)[(int64_t)ch * K + k]);
    acc[k] = dw[k] = 0.f;
  }
  const float bias = a.bias ? to_f32(((const T*)a.bias)[ch]) : 0.f;
#pragma unroll
  for (int k = 1; k < K; ++k) win[k] = row(t0 - K + k);
  int reach = reach_before(starts, t0, K);
  // acc[k] gathers the gradient of row t - (K-1) + k; a row is stored when it leaves the window
  const auto store = [&](int s, float v) {
    if (s >= t0 && s < t1) ((T*)a.dx)[((int64_t)b * a.t + s) * a.c + ch] = from_f32<T>(v);
    if (s < 0 && p == 0 && a.dstate)
      ((T*)a.dstate)[((int64_t)b * (K - 1) + s + K - 1) * a.c + ch] = from_f32<T>(v);
  };
  for (int t = t0; t < end; ++t) {
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) {
      win[k] = win[k + 1];
      acc[k] = acc[k + 1];
    }
    win[K - 1] = row(t);
    acc[K - 1] = 0.f;
    reach = starts && starts[t] ? 0 : min(reach + 1, K - 1);
    float dz = to_f32(dy[(int64_t)t * a.dy.st]);
    if (a.act) {
      float z = bias;
#pragma unroll
      for (int k = 0; k < K; ++k) z = K - 1 - k <= reach ? fmaf(w[k], win[k], z) : z;
      dz *= silu_grad(z);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      acc[k] = K - 1 - k <= reach ? fmaf(w[k], dz, acc[k]) : acc[k];
      if (t < t1) dw[k] = K - 1 - k <= reach ? fmaf(dz, win[k], dw[k]) : dw[k];
    }
    if (t < t1) db += dz;
    store(t - (K - 1), acc[0]);
  }
  // rows still in the window, with what the carried rows' gradient adds at the end
  const int at_end = end == a.t ? reach_before(starts, a.t, K) : -1;
#pragma unroll
  for (int k = 1; k < K; ++k) {
    const int s = end - K + k;
    float v = acc[k];
    if (a.dstate_out && end == a.t && (a.t == 0 || a.t - 1 - s <= at_end))
      v += to_f32(((const T*)a.dstate_out)[((int64_t)b * (K - 1) + k - 1) * a.c + ch]);
    store(s, v);
  }
  float* out = a.work + (int64_t)part * (K + 1) * a.c + ch;
#pragma unroll
  for (int k = 0; k < K; ++k) out[(int64_t)k * a.c] = dw[k];
  out[(int64_t)K * a.c] = db;
}

// Sums the pieces' parts in order.
template <int K>
__global__ __launch_bounds__(256) void seq_conv_sum_kernel(const float* work, int parts, int c, float* dw,
                                                           float* db) {
  const int ch = blockIdx.x * 256 + threadIdx.x;
  if (ch >= c) return;
  for (int k = 0; k <= K; ++k) {
    float s = 0.f;
    for (int p = 0; p < parts; ++p) s += work[((int64_t)p * (K + 1) + k) * c + ch];
    if (k < K)
      dw[(int64_t)ch * K + k] = s;
    else if (db)
      db[ch] = s;
  }
}

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

// f(T{}, integral_constant K) for the problem's type and taps.
template <int K>
struct Taps {
  static constexpr int value = K;
};
template <typename F>
hipError_t for_taps(int dtype, int k, const F& f) {
  const auto typed = [&](auto kk) {
    if (dtype == convfwd::kF32) return f(float{}, kk);
    if (dtype == convfwd::kF16) return f(_Float16{}, kk);
    return f(__bf16{}, kk);
  };
  switch (k) {
    case 1: return typed(Taps<1>{});
    case 2: return typed(Taps<2>{});
    case 3: return typed(Taps<3>{});
    case 4: return typed(Taps<4>{});
    case 5: return typed(Taps<5>{});
    case 6: return typed(Taps<6>{});
    case 7: return typed(Taps<7>{});
    default: return typed(Taps<8>{});
  }
}

int pieces_of(int t) { return t > 0 ? (t + kPiece - 1) / kPiece : 1; }

}  // namespace

int64_t conv_bwd_work_bytes(int b, int t, int c, int k) { return (int64_t)b * pieces_of(t) * (k + 1) * c * 4; }

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s) {
  const int groups = a.t > 0 ? (a.t + kGroup - 1) / kGroup : 1;
  const dim3 grid((unsigned)((a.c + 255) / 256 * a.b * groups));
  return for_taps(a.dtype, a.k, [&](auto t, auto k) {
    hipLaunchKernelGGL((seq_conv_fwd_kernel<decltype(t), decltype(k)::value>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s) {
  const int parts = a.b * pieces_of(a.t);
  return for_taps(a.dtype, a.k, [&](auto t, auto k) {
    constexpr int K = decltype(k)::value;
    if (parts > 0)
      hipLaunchKernelGGL((seq_conv_bwd_kernel<decltype(t), K>), dim3((a.c + 255) / 256 * parts), dim3(256), 0, s,
                         a);
    hipLaunchKernelGGL((seq_conv_sum_kernel<K>), dim3((a.c + 255) / 256), dim3(256), 0, s, a.work, parts, a.c,
                       a.dw, a.dbias);
    return hipGetLastError();
  });
}

hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t s) {
  return for_taps(a.dtype, a.k, [&](auto t, auto k) {
    hipLaunchKernelGGL((seq_conv_step_kernel<decltype(t), decltype(k)::value>), dim3((a.c + 255) / 256 * a.b),
                       dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace convseq
