// seq_carry.h -- the state of a recurrence h -> A h + H carried between tiles
// of one launch.
//
// A piece of rows acts on the state before it as h -> A h + H with A in [0, 1].
// A piece that holds a start forgets that state: its A is stored with the sign
// bit set (forgets()), H is its own, and selections, not products with zero,
// keep a NaN from crossing.
//
// Tiles along a sequence are handed to workgroups by a ticket counter in the
// order of the recurrence, all columns of a tile row before the next.  A tile
// publishes its (A, H) as one 64-bit word a channel, looks back over its
// predecessors' words, composing them until one is a whole state (marked as one
// that forgets), and publishes its own whole state in place of its (A, H).  A
// word that is not there yet has A's bits zero.  A waiting tile waits on tiles
// of lower tickets only; those were taken by workgroups that already run, the
// lowest of them waits for nobody, so every wait ends.  (A wait that could not
// end, in a workspace that another call overwrites, gives up after kSpins and
// puts NaN into the results.)
//
// The words are written and read with relaxed device-wide 64-bit atomics:
// value and presence travel in one access, so no fence is needed.
#pragma once

#include "seq_device.h"

namespace convseq {

constexpr uint32_t kWhole = 0x80000000u;  // A of a published state
constexpr int kSpins = 1 << 20;
constexpr int kTicketBytes = 256;

struct Carry {
  float a, h;
};

__device__ __forceinline__ bool forgets(float a) { return (int)__float_as_uint(a) < 0; }

// first, then second
__device__ __forceinline__ Carry compose(Carry first, Carry second) {
  return forgets(second.a) ? second : Carry{first.a * second.a, fmaf(second.a, first.h, second.h)};
}
__device__ __forceinline__ float apply(Carry c, float h) { return forgets(c.a) ? c.h : fmaf(c.a, h, c.h); }

__device__ __forceinline__ void publish(uint64_t* word, Carry c) {
  const uint32_t a = max(__float_as_uint(c.a), 1u);  // A = 0 as the smallest number: bits zero mean absent
  __hip_atomic_store(word, (uint64_t)__float_as_uint(c.h) << 32 | a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* word) {
  return __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The states before tile `tile` of V channels a lane, from the words of the
// tiles before it: `words` is tile 0's, tiles are `step` words apart.  Called
// by one whole wave.
//
// It walks back until every lane has seen a whole state, then applies the tiles
// from there in the order of the recurrence.  A whole state was itself made by
// applying its tile to the state before it, so where the walk ended, which
// depends on timing, does not show in a single bit of the result.
template <int V>
__device__ __forceinline__ void look_back(const uint64_t* words, int64_t step, int tile, float (&state)[V]) {
  constexpr int kAhead = 4;  // words read at once
  uint64_t w[kAhead][V];
  bool done[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    state[i] = 0.f;
    done[i] = false;
  }
  int k = tile - 1;  // nearest tile not yet taken
  int spins = 0;
  for (;;) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) w[j][i] = peek(words + (int64_t)max(k - j, 0) * step + i);
    int taken = 0;
    bool all = false;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      bool there = true, end = true;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        there &= done[i] || (uint32_t)w[j][i] != 0u;
        end &= done[i] || (int)(uint32_t)w[j][i] < 0;
      }
      if (taken == j && !all && k - j >= 0 && __all(there)) {
        taken = j + 1;
        all = __all(end);
#pragma unroll
        for (int i = 0; i < V; ++i) done[i] |= (int)(uint32_t)w[j][i] < 0;
      }
    }
    k -= taken;
    if (all) break;
    if (taken == 0) {
      if (++spins > kSpins) {
#pragma unroll
        for (int i = 0; i < V; ++i) state[i] = __uint_as_float(0x7fc00000u);
        return;
      }
      __builtin_amdgcn_s_sleep(1);
    }
  }
  // all words of tiles k+1 .. tile-1 are there, and the first is whole in some
  // lane, so that every lane meets a whole state on the way up
  for (++k; k < tile; k += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) w[j][i] = peek(words + (int64_t)min(k + j, tile - 1) * step + i);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k + j < tile)
#pragma unroll
        for (int i = 0; i < V; ++i)
          state[i] = apply(Carry{__uint_as_float((uint32_t)w[j][i]), __uint_as_float((uint32_t)(w[j][i] >> 32))}, state[i]);
  }
}

// Zero for the ticket and the words; a kernel rather than a memset, which a
// captured graph has to be able to replay.
static __global__ __launch_bounds__(256) void carry_clear_kernel(uint4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = make_uint4(0, 0, 0, 0);
}
inline hipError_t carry_clear(void* work, int64_t bytes, hipStream_t s) {
  const int64_t n = bytes / 16, b = (n + 255) / 256;
  hipLaunchKernelGGL(carry_clear_kernel, dim3((unsigned)(b < 2048 ? b : 2048)), dim3(256), 0, s, (uint4*)work, n);
  return hipGetLastError();
}

}  // namespace convseq
