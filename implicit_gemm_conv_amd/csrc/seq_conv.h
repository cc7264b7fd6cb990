// seq_conv.h -- device helpers shared by the causal depthwise convolution's
// kernels.
//
//   z_t = bias + sum_k w_k X(t - (K-1) + k),   y = z or z * sigmoid(z)
//
// X is x, below row 0 the carried rows, and zero across a start.  How far back
// row t may look, reach(t) = min(K-1, t - (last start <= t)), depends on (b, t)
// alone, so it is the same for every lane of a wave: a tap j rows back counts
// iff j <= reach(t), and is selected, not multiplied, away.
#pragma once

#include "seq_device.h"

namespace convseq {

__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }
__device__ __forceinline__ float silu_grad(float z) {
  const float s = sigmoid(z);
  return s * fmaf(z, 1.f - s, 1.f);
}

// reach(t - 1) of the row before t (rows before row 0 reach everything).
__device__ __forceinline__ int reach_before(const uint8_t* starts, int t, int k) {
  if (!starts) return k - 1;
  for (int j = 1; j < k && t - j >= 0; ++j)
    if (starts[t - j]) return j - 1;
  return k - 1;
}

// V channels of X at row s, `offset` bytes into the row: x, or below row 0 the carried rows (zero if there are none).
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> row_at(const T* x, int64_t st, const T* state, int s, int k, int c,
                                             uint32_t offset) {
  Pack<T, V> v;
  if (s >= 0) return load_at<Pack<T, V>>(x + (int64_t)s * st, offset);
  if (state) return load_at<Pack<T, V>>(state + (int64_t)(s + k - 1) * c, offset);
#pragma unroll
  for (int i = 0; i < V; ++i) v.set(i, 0.f);
  return v;
}

template <int K>
struct Taps {
  static constexpr int value = K;
};
// f(Taps<k>) for the problem's taps.
template <typename F>
hipError_t for_taps(int k, const F& f) {
  switch (k) {
    case 1: return f(Taps<1>{});
    case 2: return f(Taps<2>{});
    case 3: return f(Taps<3>{});
    case 4: return f(Taps<4>{});
    case 5: return f(Taps<5>{});
    case 6: return f(Taps<6>{});
    case 7: return f(Taps<7>{});
    default: return f(Taps<8>{});
  }
}

}  // namespace convseq
