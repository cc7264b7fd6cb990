// seq_carry.h -- the state of a recurrence h -> A h + H carried between tiles
// of one launch.
//
// A piece of rows acts on the state before it as h -> A h + H with A in (0, 1]:
// a product that fp32 would round to zero is its smallest number (positive()).
// A piece that holds a start forgets that state: its A is stored with the sign
// bit set (forgets()), H is its own, and selections, not products with zero,
// keep a NaN from crossing.
//
// The tiles of a column (64 V channels of one sequence) are handed to workgroups
// by the column's ticket counter, in the order of the recurrence.  A tile
// publishes its (A, H) as one 64-bit word a channel, looks back over its
// predecessors, applies their steps from the nearest whole state on, and
// publishes its own whole state (a word that forgets) in place of its (A, H).
// A waiting tile waits on lower tickets of its column only; those were taken by
// workgroups that already run, the lowest of them waits for nobody, so every
// wait ends.  (A wait that could not end, in a workspace that another call
// overwrites, gives up after kSpins and puts NaN into the results.)  One counter
// for all columns would cost 3 us where a few hundred workgroups start at once.
//
// Words and flags are written and read with relaxed device-wide atomics, in no
// order between them.  A word says by itself, in one access, whether it is there
// (A's bits are zero until then) and whether it is a whole state (A's sign), so no
// fence is needed: a reader that wants a whole state waits until the word is one,
// whatever the flag said, since the flag may be seen before the word that it
// announces and the tile's step, published earlier, still be in its place.  The
// flags, one a tile and column, only say where to look: a wave reads those of 64 tiles at once, and polling them
// instead of the words keeps the waiting off the memory the tiles stream
// through (words of 32 tiles polled by all waves took an early 1x65539x1024 bf16
// forward 174 us, 4 at a time by one wave 155).
#pragma once

#include "seq_device.h"

namespace convseq {

constexpr uint32_t kWhole = 0x80000000u;  // A of a published state
constexpr int kSpins = 1 << 20;
constexpr int kTicketBytes = 64;  // a column's counter, a cache line of its own

struct Carry {
  float a, h;
};

__device__ __forceinline__ bool forgets(float a) { return (int)__float_as_uint(a) < 0; }

// first, then second
__device__ __forceinline__ Carry compose(Carry first, Carry second) {
  return forgets(second.a) ? second : Carry{positive(first.a * second.a), fmaf(second.a, first.h, second.h)};
}
__device__ __forceinline__ float apply(Carry c, float h) { return forgets(c.a) ? c.h : fmaf(c.a, h, c.h); }

__device__ __forceinline__ void publish(uint64_t* word, Carry c) {
  // A is positive or has its sign set: bits zero mean absent
  __hip_atomic_store(word, (uint64_t)__float_as_uint(c.h) << 32 | __float_as_uint(c.a), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* word) {
  return __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What a launch's tiles share, in its workspace: a ticket a column, a flag a
// column and tile, a word a tile and lane channel.
struct CarrySpace {
  char* tickets;
  uint32_t* flags;  // [columns][tiles]
  uint64_t* words;  // [tiles][columns][lane channels]
};
__host__ __device__ inline int64_t carry_head_bytes(int64_t tiles, int64_t columns) {
  return columns * kTicketBytes + (tiles * columns * 4 + 15) / 16 * 16;
}
// Bytes for `tiles` tiles that publish and `columns` columns of `width` channels.
inline int64_t carry_bytes(int64_t tiles, int64_t columns, int width) {
  return carry_head_bytes(tiles, columns) + tiles * columns * width * 8;
}
__device__ __forceinline__ CarrySpace carry_space(void* work, int64_t tiles, int64_t columns) {
  char* p = (char*)work;
  return CarrySpace{p, (uint32_t*)(p + columns * kTicketBytes), (uint64_t*)(p + carry_head_bytes(tiles, columns))};
}
// The workgroup's place in the order of its column.
__device__ __forceinline__ int take_ticket(void* work, int column, int* shared) {
  if (threadIdx.x == 0)
    *shared = __hip_atomic_fetch_add((int*)((char*)work + (int64_t)column * kTicketBytes), 1, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
  lds_barrier();
  return __builtin_amdgcn_readfirstlane(*shared);
}

// The words a workgroup gathers at once, and how many tiles it has to apply.
constexpr int kEach = 2;  // of a wave
constexpr int kFold = 4;
template <int V, int WAVES>
struct Gathered {
  uint64_t words[WAVES * kEach][64 * V];
  static_assert(WAVES * kEach % kFold == 0, "whole groups");
  int span;
};

__device__ __forceinline__ void raise_flag(uint32_t* flag, uint32_t v) {
  __hip_atomic_store(flag, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The states before tile `tile` of V channels a lane, in the waves for which
// `fold` is set (one wave); called by all waves of a workgroup.  `words` is tile
// 0's first word of the column, tiles are `step` words apart; `flags` is tile 0's flag:
// 1 for a published step, 2 for a whole state.
//
// The tiles from the nearest whole state on are applied in the order of the
// recurrence.  A whole state was itself made by applying its tile to the state
// before it, so which one was the nearest, a matter of timing, does not show in
// a single bit of the result.
template <int V, int WAVES>
__device__ __forceinline__ void look_back(const uint64_t* words, int64_t step, const uint32_t* flags, int tile, int wave,
                                          int lane, bool fold, Gathered<V, WAVES>& sh, float (&state)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) state[i] = 0.f;
  if (fold) {
    int span = 0;  // tiles seen, none of them whole, nearest first
    for (int spins = 0;;) {
      const int k = tile - 1 - span - lane;
      const uint32_t f = k >= 0 ? __hip_atomic_load(flags + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
      const uint64_t there = __ballot(f != 0u), whole = __ballot(f == 2u);
      const int n = there == ~0ull ? 64 : __builtin_ctzll(~there);  // so many in a row
      const int d = whole ? __builtin_ctzll(whole) : 64;
      if (d < n) {
        span += d + 1;
        break;
      }
      span += n;
      if (n == 0) {
        if (++spins > kSpins) {
          span = -1;
          break;
        }
        __builtin_amdgcn_s_sleep(1);
      }
    }
    if (lane == 0) sh.span = span;
  }
  lds_barrier();
  const int span = __builtin_amdgcn_readfirstlane(sh.span);
  const bool lost = span < 0;
  const int oldest = tile - max(span, 0);  // the one that has to be a whole state
  for (int from = oldest; from < tile; from += WAVES * kEach) {
    const int count = min(tile - from, WAVES * kEach);
    // a scalar mask: tests in the lanes spill the forward kernel's registers (137 us
    // instead of 124 for 1x65539x1024 bf16)
    const uint32_t need = from == oldest && wave == 0 ? kWhole : ~0u;
    uint64_t w[kEach][V];
    for (int spins = 0;;) {
      bool there = true;
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (j * WAVES + wave < count) {
#pragma unroll
          for (int i = 0; i < V; ++i) w[j][i] = peek(words + (int64_t)(from + j * WAVES + wave) * step + (uint32_t)(lane * V + i));
        }
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (j * WAVES + wave < count) {
#pragma unroll
          for (int i = 0; i < V; ++i) there &= ((uint32_t)w[j][i] & (j == 0 ? need : ~0u)) != 0u;
        }
      if (__all(there)) break;
      if (++spins > kSpins) {  // gives up: a whole state of NaN
#pragma unroll
        for (int j = 0; j < kEach; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) w[j][i] = 0x7fc0000080000000ull;
        break;
      }
      __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)  // past the last tile: a step that changes nothing
        sh.words[j * WAVES + wave][lane * V + i] = j * WAVES + wave < count ? w[j][i] : 0x3f800000ull;
    lds_barrier();
    if (fold)
      for (int slot = 0; slot < count; slot += kFold) {
        uint64_t v[kFold][V];  // read together, applied one after the other
#pragma unroll
        for (int j = 0; j < kFold; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) v[j][i] = sh.words[slot + j][lane * V + i];
#pragma unroll
        for (int j = 0; j < kFold; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i)
            state[i] = apply(Carry{__uint_as_float((uint32_t)v[j][i]), __uint_as_float((uint32_t)(v[j][i] >> 32))}, state[i]);
      }
    lds_barrier();
  }
  if (lost)
#pragma unroll
    for (int i = 0; i < V; ++i) state[i] = __uint_as_float(0x7fc00000u);
}

// Zero for tickets, flags and words; a kernel rather than a memset, which a
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
