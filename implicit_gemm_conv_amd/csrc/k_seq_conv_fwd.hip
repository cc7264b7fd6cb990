// k_seq_conv_fwd.hip -- causal depthwise convolution along a sequence, forward.
//
// A wave takes 16 rows by 64 V channels, a lane V channels of those: it reads
// its rows and the K-1 before them once, all loads in flight together, and
// makes K multiply-adds a value from registers.  The 4 waves of a workgroup
// take 4 consecutive row groups of the same channels, so that 3 of 4 waves find
// their K-1 earlier rows in the cache of their own compute unit.  Memory bound:
// x read once, y written once; 1x32771x1024 fp16 takes 27.1 us (5.0 TB/s), and
// 4x4096x2048 bf16 with 8 bits kept 38 to 40 us (4.2 to 4.5 TB/s).  V is 2 where C and
// the buffers' alignment allow pairs, else 1.  With 1, 2 and 4 channels a lane, calls back
// to back on inputs in turn: 30.0, 28.7 and 32.2 us, and 36.3, 35.7 and 37.5 (at 4 the
// registers leave 5 waves a SIMD instead of 8).
#include "seq_conv.h"

namespace convseq {

namespace {

constexpr int kWaves = 4;

template <typename T, int K, int V>
__global__ __launch_bounds__(kWaves * 64) void seq_conv_fwd_kernel(ConvArgs a, int cols, int blocks) {
  typedef Pack<T, V> P;
  const int lane = threadIdx.x & 63;
  const int groups = max(1, (a.t + kGroup - 1) / kGroup);
  const int id = blockIdx.x / cols, b = id / blocks;
  const int g = __builtin_amdgcn_readfirstlane(id % blocks * kWaves + (threadIdx.x >> 6));
  if (g >= groups) return;
  const int chs = ((int)(blockIdx.x % cols) * 64 + lane) * V;
  const bool own = chs < a.c;
  const int ch = min(chs, a.c - V);  // lanes past the last channel read it again
  const int t0 = g * kGroup, n = min(a.t - t0, kGroup);
  const uint32_t offset = (uint32_t)ch * sizeof(T);
  const T* x = (const T*)a.x.p + b * a.x.sb;
  const T* state = a.state ? (const T*)a.state + (int64_t)b * (K - 1) * a.c : nullptr;
  const uint8_t* starts = a.starts ? a.starts + (int64_t)b * a.t : nullptr;

  P raw[K - 1 + kGroup];  // rows t0 - (K-1) on
  if (t0 > 0) {           // K - 1 < 16 rows lie before it
#pragma unroll
    for (int j = 0; j < K - 1; ++j) raw[j] = load_at<P>(x + (int64_t)(t0 - (K - 1) + j) * a.x.st, offset);
  } else {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) raw[j] = row_at<T, V>(x, a.x.st, state, j - (K - 1), K, a.c, offset);
  }
  if (n > 0) {
    uint32_t from = offset;
    renew(from);
    RowWalk rows(x + (int64_t)t0 * a.x.st, a.x.st * (int64_t)sizeof(T));
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {  // rows past the last repeat it
      raw[K - 1 + j] = rows.load<P>(from);
      rows.step(j + 1 < n);
    }
  }
  uint32_t first = 0;  // bit j: row t0 + j begins a sequence
  int reach = K - 1;
  if (starts) {
    first = (uint32_t)__ballot(lane < n && starts[t0 + lane]);
    reach = reach_before(starts, t0, K);
  }
  float w[K][V], bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][i] = to_f32(((const T*)a.w)[(int64_t)(ch + i) * K + k]);
    bias[i] = a.bias ? to_f32(((const T*)a.bias)[ch + i]) : 0.f;
  }

  if (a.kept.q && n > 0 && own)
    keep_group<T, V>(*(const P(*)[kGroup])(raw + K - 1), n, a.kept, (int64_t)b * groups + g, a.c, ch);

  T* y = (T*)a.y + ((int64_t)b * a.t + t0) * a.c;
  // `plain`: 16 rows that all reach K - 1 rows back, with or without the activation
  const auto run = [&](auto plain, auto activated) {
    constexpr bool masked = !decltype(plain)::value;
    const bool act = masked ? a.act != 0 : decltype(activated)::value;
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (!masked || j < n) {
        if (masked) reach = first >> j & 1 ? 0 : min(reach + 1, K - 1);
        P out;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float z = bias[i];
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float sum = fmaf(w[k][i], raw[j + k].get(i), z);
            z = !masked || K - 1 - k <= reach ? sum : z;
          }
          out.set(i, act ? silu(z) : z);
        }
        if (own) store_at(y + (int64_t)j * a.c, offset, out);
      }
  };
  if (n < kGroup || first || reach < K - 1)
    run(No{}, No{});
  else if (a.act)
    run(Yes{}, Yes{});
  else
    run(Yes{}, No{});

  if (a.state_out && g == groups - 1 && own) {
    T* out = (T*)a.state_out + (int64_t)b * (K - 1) * a.c;
    reach = reach_before(starts, a.t, K);
    for (int j = 0; j < K - 1; ++j) {
      const int s = a.t - (K - 1) + j;
      P v = row_at<T, V>(x, a.x.st, state, s, K, a.c, offset);
      if (a.t > 0 && a.t - 1 - s > reach)
#pragma unroll
        for (int i = 0; i < V; ++i) v.set(i, 0.f);
      store_at(out + (int64_t)j * a.c, offset, v);
    }
  }
}

template <typename T, int V>
hipError_t run(const ConvArgs& a, hipStream_t s) {
  const int cols = (a.c + 64 * V - 1) / (64 * V);
  const int blocks = a.t > 0 ? (a.t + kWaves * kGroup - 1) / (kWaves * kGroup) : 1;
  return for_taps(a.k, [&](auto k) {
    hipLaunchKernelGGL((seq_conv_fwd_kernel<T, decltype(k)::value, V>), dim3((unsigned)(cols * a.b * blocks)),
                       dim3(kWaves * 64), 0, s, a, cols, blocks);
    return hipGetLastError();
  });
}

template <typename T, int V>
hipError_t run_wide(const ConvArgs& a, hipStream_t s) {
  constexpr int e = sizeof(T), bytes = V * e;
  const uintptr_t at = (uintptr_t)a.y | (uintptr_t)a.state | (uintptr_t)a.state_out | (uintptr_t)a.kept.e * e;
  return a.c % V == 0 && pieces(a.x, bytes, e) && at % bytes == 0 ? run<T, V>(a, s) : run<T, 1>(a, s);
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s) {
  if (a.dtype == convfwd::kF32) return run_wide<float, 2>(a, s);
  if (a.dtype == convfwd::kF16) return run_wide<_Float16, 2>(a, s);
  return run_wide<__bf16, 2>(a, s);
}

}  // namespace convseq
