// k_seq_keep8.hip -- a (B, T, C) tensor into 8 bits and back.  Groups of 16
// consecutive rows of one channel share a power of two: down a channel values
// are of one scale where channels of one row are not, and neighbouring lanes
// hold neighbouring channels, so the largest of a group needs no exchange
// between lanes.  A lane takes V channels of one group: 16 row pieces of V
// values on one side, two runs of 8 V bytes on the other.  Memory bound: 8x8192x2048
// bf16, calls back to back on inputs in turn, takes 73 us to pack and 79 to unpack (5.6
// and 5.2 TB/s, where a copy reaches 5.1 to 5.3); into new memory a pack takes 90 at the
// median, and what was just packed comes back in 65, part of it from the last-level
// cache.  With 1, 2 and 4 channels a lane a pack takes 71, 73 and 75 us, apart by no more
// than the spread, and of 4x4096x2048, which stays in the cache, 19.9, 17.8 and 19.6; an
// unpack takes 79, 75 and 79.
#include "seq_device.h"

namespace convseq {

namespace {

// Where a lane of the grid works: channels ch on, rows t0 .. t0 + n - 1 of batch
// b.  Lanes are dealt over all (group, V channels) pairs in a row, so that none
// idles behind a channel count that 64 V does not divide (65 channels in waves of
// their own would leave half the lanes without work).
struct Place {
  int ch, b, t0, n, part;  // part: b and the group as one index
};
template <int V>
__device__ __forceinline__ bool place(int parts, int t, int c, int groups, Place* p) {
  const uint32_t pieces = (uint32_t)c / V;  // of a group
  const int64_t first = ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 64;
  // the wave's first piece by wave-uniform division, the lane's from there
  const uint32_t at = (uint32_t)(first % pieces) + (threadIdx.x & 63), step = at / pieces;
  p->part = (int)(first / pieces) + (int)step;
  p->ch = (int)(at - step * pieces) * V;
  p->b = p->part / groups;
  p->t0 = (p->part - p->b * groups) * kGroup;
  p->n = min(t - p->t0, kGroup);
  return p->part < parts;
}

template <typename T, int V>
__global__ __launch_bounds__(256) void pack8_kernel(int parts, int t, int c, int groups, Rows x, Kept k) {
  Place p;
  if (!place<V>(parts, t, c, groups, &p)) return;
  typedef Pack<T, V> P;
  const T* in = (const T*)x.p + p.b * x.sb + (int64_t)p.t0 * x.st + p.ch;
  P raw[kGroup];
#pragma unroll
  for (int j = 0; j < kGroup; ++j) raw[j] = *(const P*)(in + (int64_t)min(j, p.n - 1) * x.st);
  keep_group<T, V>(raw, p.n, k, p.part, c, p.ch);
}

template <typename T, int V>
__global__ __launch_bounds__(256) void unpack8_kernel(int parts, int t, int c, int groups, Kept k, T* out) {
  Place p;
  if (!place<V>(parts, t, c, groups, &p)) return;
  typedef Pack<T, V> P;
  Half<V> q[2];
  float scale[V];
#pragma unroll
  for (int h = 0; h < 2; ++h) q[h] = half_group<V>(k, p.part, h, c, p.ch);
  group_scales<V>(k, p.part, c, p.ch, scale);
  T* to = out + ((int64_t)p.b * t + p.t0) * c + p.ch;
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < p.n) {
      P v;
#pragma unroll
      for (int i = 0; i < V; ++i) v.set(i, q[j / 8].get(i, j % 8) * scale[i]);
      *(P*)(to + (int64_t)j * c) = v;
    }
}

template <int V>
unsigned blocks(int64_t parts, int c) {
  return (unsigned)((parts * (c / V) + 255) / 256);
}

template <typename T, int V>
hipError_t pack_as(int b, int t, int c, const Rows& x, const Kept& k, hipStream_t s) {
  const int groups = (t + kGroup - 1) / kGroup;
  hipLaunchKernelGGL((pack8_kernel<T, V>), dim3(blocks<V>((int64_t)b * groups, c)), dim3(256), 0, s, b * groups, t, c,
                     groups, x, k);
  return hipGetLastError();
}
template <typename T, int V>
hipError_t unpack_as(int b, int t, int c, const Kept& k, void* out, hipStream_t s) {
  const int groups = (t + kGroup - 1) / kGroup;
  hipLaunchKernelGGL((unpack8_kernel<T, V>), dim3(blocks<V>((int64_t)b * groups, c)), dim3(256), 0, s, b * groups, t, c,
                     groups, k, (T*)out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pack8(int b, int t, int c, int dtype, const Rows& x, const Kept& k, hipStream_t s) {
  if (dtype == convfwd::kF32)
    return c % 2 == 0 && pieces(x, 8, 4) && (uintptr_t)k.e % 2 == 0 ? pack_as<float, 2>(b, t, c, x, k, s) : pack_as<float, 1>(b, t, c, x, k, s);
  const bool wide = c % 2 == 0 && pieces(x, 4, 2) && (uintptr_t)k.e % 2 == 0;
  if (dtype == convfwd::kF16) return wide ? pack_as<_Float16, 2>(b, t, c, x, k, s) : pack_as<_Float16, 1>(b, t, c, x, k, s);
  return wide ? pack_as<__bf16, 2>(b, t, c, x, k, s) : pack_as<__bf16, 1>(b, t, c, x, k, s);
}

hipError_t launch_unpack8(int b, int t, int c, int dtype, const Kept& k, void* out, hipStream_t s) {
  if (dtype == convfwd::kF32)
    return c % 2 == 0 && (uintptr_t)out % 8 == 0 && (uintptr_t)k.e % 2 == 0 ? unpack_as<float, 2>(b, t, c, k, out, s)
                                                 : unpack_as<float, 1>(b, t, c, k, out, s);
  const bool wide = c % 4 == 0 && (uintptr_t)out % 8 == 0 && (uintptr_t)k.e % 4 == 0;
  if (dtype == convfwd::kF16) return wide ? unpack_as<_Float16, 4>(b, t, c, k, out, s) : unpack_as<_Float16, 1>(b, t, c, k, out, s);
  return wide ? unpack_as<__bf16, 4>(b, t, c, k, out, s) : unpack_as<__bf16, 1>(b, t, c, k, out, s);
}

}  // namespace convseq
