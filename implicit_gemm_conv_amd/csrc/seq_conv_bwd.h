// seq_conv_bwd.h -- causal depthwise convolution along a sequence, backward.
//
//   dz_t = dy_t act'(z_t)  (z_t computed again from x)
//   dx_s = sum_j w_{K-1-j} dz_{s+j},   dw_k = sum_t dz_t X(t - (K-1) + k),   dbias = sum_t dz_t
//
// A lane walks down G groups of 16 rows of V channels with the last K values of
// X and the K unfinished rows of dx in registers, loading 8 rows while it works on
// the 8 before: row t gives dz_t to the K rows it looked at, and row t - (K-1) is
// then complete and stored.  It ends with the
// K-1 rows after its own, for what they send back.  dw and dbias gather in
// registers, are added over the 4 waves of the workgroup (4 consecutive pieces
// of the same channels) in LDS and over the workgroups by a second kernel, both
// in a fixed order.  Memory bound: dy and x (or its 8 bits) read once, dx
// written once; 4x4096x2048 bf16 from 8 bits takes 44.8 us, the vector ALU busy
// 60% of it.
#pragma once

#include "seq_conv.h"

namespace convseq {

namespace {

constexpr int kWaves = 4;
constexpr int kChunk = 8;  // rows loaded at once

// Rows in flight: dy, x or its 8 bits, and which of them begin a sequence.
template <typename T, int V, bool KEPT>
struct Chunk {
  Pack<T, V> dy[kChunk], x[KEPT ? 1 : kChunk];
  Half<V> q;
  float scale[V];
  uint32_t first;
};

// Four waves a SIMD (128 registers) where the windows leave room for it.  With the bound
// at 4 and at 2 waves (which leaves the choice to the registers), 4x4096x2048 bf16, silu,
// calls back to back with their sums, from x / from 8 bits:
//   K        1-2        3            4            5            6            8
//   4 waves  44 / 39    45 / 42      47 / 45      50 / 58      64 / 80      170 / 177 us
//   2 waves  44 / 39    45 / 54      47 / 57      58 / 59      57 / 61      67 / 73 us
// The rule takes the better side at V = 2 but for K = 5 from x.
template <typename T, int K, int V, bool KEPT>
__global__ __launch_bounds__(kWaves * 64, K * V <= 8 ? 4 : 2) void seq_conv_bwd_kernel(ConvArgs a, int cols, int blocks, int per) {
  typedef Pack<T, V> P;
  __shared__ float sums[kWaves][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = (a.t + kGroup - 1) / kGroup;
  const int id = blockIdx.x / cols, b = __builtin_amdgcn_readfirstlane(id / blocks);
  const int piece = __builtin_amdgcn_readfirstlane(id % blocks * kWaves + wave);
  const int chs = ((int)(blockIdx.x % cols) * 64 + lane) * V;
  const bool own = chs < a.c;
  const int ch = min(chs, a.c - V);  // lanes past the last channel read it again
  const bool ragged = (int)(blockIdx.x % cols + 1) * 64 * V > a.c;
  // rows t0 .. t1 - 1 are this lane's; pieces past the end have none
  const int t0 = (int)min((int64_t)a.t, (int64_t)piece * per * kGroup);
  const bool here = t0 < a.t || piece == 0;
  const int t1 = min(a.t - t0, per * kGroup) + t0;
  const uint32_t offset = (uint32_t)ch * sizeof(T);
  const T* x = (const T*)a.x.p + b * a.x.sb;
  const T* dy = (const T*)a.dy.p + b * a.dy.sb;
  const T* state = a.state ? (const T*)a.state + (int64_t)b * (K - 1) * a.c : nullptr;
  const uint8_t* starts = a.starts ? a.starts + (int64_t)b * a.t : nullptr;

  float w[K][V], bias[V], win[K][V], acc[K][V], dw[K + 1][V];  // dw[K]: dbias
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      w[k][i] = to_f32(((const T*)a.w)[(int64_t)(ch + i) * K + k]);
      win[k][i] = acc[k][i] = dw[k][i] = 0.f;
    }
    bias[i] = a.bias ? to_f32(((const T*)a.bias)[ch + i]) : 0.f;
    dw[K][i] = 0.f;
  }

  if (here) {
    // X of rows t0 - (K-1) .. t0 - 1 into win[1 ..]
#pragma unroll
    for (int k = 1; k < K; ++k) {
      const int s = t0 - K + k;
      if (!KEPT || s < 0) {
        const P v = row_at<T, V>(x, a.x.st, state, s, K, a.c, offset);
#pragma unroll
        for (int i = 0; i < V; ++i) win[k][i] = v.get(i);
      }
    }
    if (KEPT && t0 > 0) {
      const int64_t at = (int64_t)b * groups + t0 / kGroup - 1;
      const Half<V> q = half_group<V>(a.kept, at, 1, a.c, ch);  // rows 8 .. 15, K - 1 <= 7
      float scale[V];
      group_scales<V>(a.kept, at, a.c, ch, scale);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 1; k < K; ++k) win[k][i] = q.get(i, 8 - K + k) * scale[i];
    }
    int reach = reach_before(starts, t0, K);
    // row s of dx is complete; below row 0 it is a carried row's gradient
    const auto store = [&](int s, const float(&v)[V]) {
      P out;
#pragma unroll
      for (int i = 0; i < V; ++i) out.set(i, v[i]);
      if (!own) return;
      if (s >= t0 && s < t1) store_at((T*)a.dx + ((int64_t)b * a.t + s) * a.c, offset, out);
      if (s < 0 && piece == 0 && a.dstate)
        store_at((T*)a.dstate + ((int64_t)b * (K - 1) + s + K - 1) * a.c, offset, out);
    };

    const int end = min(a.t, t1 + K - 1);
    Chunk<T, V, KEPT> now, next;
    const auto load = [&](int g0, Chunk<T, V, KEPT>& to) {
      const int n = min(end - g0, kChunk);
      uint32_t from = offset;
      renew(from);
      RowWalk wy(dy + (int64_t)g0 * a.dy.st, a.dy.st * (int64_t)sizeof(T));
      RowWalk wx(x + (int64_t)g0 * a.x.st, a.x.st * (int64_t)sizeof(T));
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {  // rows past the last repeat it
        to.dy[j] = wy.load<P>(from);
        if (!KEPT) to.x[j] = wx.load<P>(from);
        wy.step(j + 1 < n);
        wx.step(j + 1 < n);
      }
      if (KEPT) {
        const int64_t at = (int64_t)b * groups + g0 / kGroup;
        to.q = half_group<V>(a.kept, at, g0 / kChunk % 2, a.c, ch);
        group_scales<V>(a.kept, at, a.c, ch, to.scale);
      }
      to.first = starts ? (uint32_t)__ballot(lane < n && starts[g0 + lane]) : 0u;
    };
    if (t0 < end) load(t0, next);
    for (int g0 = t0; g0 < end; g0 += kChunk) {
      now = next;
      if (g0 + kChunk < end) load(g0 + kChunk, next);
      const bool mine = g0 < t1;  // else the rows after the piece, K - 1 of them at most
      const int n = min(end - g0, kChunk);
      const uint32_t first = now.first;
      // `plain`: 8 rows of the piece that all reach K - 1 rows back, in a wave with all its
      // channels, with or without the activation
      const auto run = [&](auto plain, auto activated) {
        constexpr bool masked = !decltype(plain)::value;
        const bool act = masked ? a.act != 0 : decltype(activated)::value;
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
          if (!masked || j < n) {
            if (masked) reach = first >> j & 1 ? 0 : min(reach + 1, K - 1);
            const auto live = [&](int k) { return !masked || K - 1 - k <= reach; };
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
              for (int k = 0; k + 1 < K; ++k) {
                win[k][i] = win[k + 1][i];
                acc[k][i] = acc[k + 1][i];
              }
              win[K - 1][i] = KEPT ? now.q.get(i, j) * now.scale[i] : now.x[j].get(i);
              float dz = now.dy[j].get(i);
              if (act) {
                float z = bias[i];
#pragma unroll
                for (int k = 0; k < K; ++k) z = live(k) ? fmaf(w[k][i], win[k][i], z) : z;
                dz *= silu_grad(z);
              }
#pragma unroll
              for (int k = 0; k + 1 < K; ++k) acc[k][i] = live(k) ? fmaf(w[k][i], dz, acc[k][i]) : acc[k][i];
              acc[K - 1][i] = w[K - 1][i] * dz;
              if (!masked || mine) {
#pragma unroll
                for (int k = 0; k < K; ++k) dw[k][i] = live(k) ? fmaf(dz, win[k][i], dw[k][i]) : dw[k][i];
                dw[K][i] += dz;
              }
            }
            if (masked) {
              store(g0 + j - (K - 1), acc[0]);
            } else if (j >= K - 1 || g0 > t0) {  // the row it looked back to is the piece's
              P out;
#pragma unroll
              for (int i = 0; i < V; ++i) out.set(i, acc[0][i]);
              uint32_t to = offset;
              renew(to);
              RowWalk((T*)a.dx + ((int64_t)b * a.t + g0 + j - (K - 1)) * a.c, 0).store(to, out);
            }
            // row by row: rows worked on together cost registers
            if (!masked) __builtin_amdgcn_sched_barrier(0);
          }
      };
      if (!mine || n < kChunk || first || reach < K - 1 || ragged || (t0 == 0 && a.dstate))
        run(No{}, No{});
      else if (a.act)
        run(Yes{}, Yes{});
      else
        run(Yes{}, No{});
    }
    // rows still in the window, and what the carried rows' gradient adds at the end of the sequence
    const int at_end = end == a.t ? reach_before(starts, a.t, K) : 0;
#pragma unroll
    for (int k = 1; k < K; ++k) {
      const int s = end - K + k;
      if (a.dstate_out && end == a.t && (a.t == 0 || a.t - 1 - s <= at_end)) {
        const P v = load_at<P>((const T*)a.dstate_out + ((int64_t)b * (K - 1) + k - 1) * a.c, offset);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[k][i] += v.get(i);
      }
      store(s, acc[k]);
    }
  }

  float* part = a.work + (int64_t)id * (K + 1) * a.c + ch;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][lane * V + i] = dw[k][i];
    lds_barrier();
    if (wave == 0 && own)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < kWaves; ++u) s += sums[u][lane * V + i];
        part[(int64_t)k * a.c + i] = s;
      }
    lds_barrier();
  }
}

// dw and dbias from the workgroups' parts: 32 channels of one tap a workgroup (the
// taps along the grid's y: along x, with 2^21 groups of channels, they would pass
// its 2^32 threads), 32 threads a channel that each add every 32nd part, then the threads' sums in order.
template <int K>
__global__ __launch_bounds__(1024) void seq_conv_sum_kernel(const float* work, int64_t parts, int c, float* dw, float* db) {
  __shared__ float s[32][33];
  const int k = blockIdx.y;
  const int ch = (int)blockIdx.x * 32 + (threadIdx.x & 31), turn = threadIdx.x >> 5;
  float v = 0.f;
  if (ch < c)
    for (int64_t p = turn; p < parts; p += 32) v += work[(p * (K + 1) + k) * c + ch];
  s[turn][threadIdx.x & 31] = v;
  __syncthreads();
  if (turn == 0 && ch < c) {
    v = 0.f;
    for (int j = 0; j < 32; ++j) v += s[j][threadIdx.x];
    if (k < K)
      dw[(int64_t)ch * K + k] = v;
    else if (db)
      db[ch] = v;
  }
}

template <typename T, int V>
hipError_t run(const ConvArgs& a, hipStream_t s) {
  const int cols = (a.c + 64 * V - 1) / (64 * V);
  const int per = conv_bwd_groups(a.b, a.t, a.c);
  const int blocks = conv_bwd_blocks(a.t, per);
  const int64_t parts = (int64_t)a.b * blocks;
  return for_taps(a.k, [&](auto k) {
    constexpr int K = decltype(k)::value;
    const dim3 grid((unsigned)(cols * parts)), block(kWaves * 64);
    if (parts > 0) {
      if (a.kept.q)
        hipLaunchKernelGGL((seq_conv_bwd_kernel<T, K, V, true>), grid, block, 0, s, a, cols, blocks, per);
      else
        hipLaunchKernelGGL((seq_conv_bwd_kernel<T, K, V, false>), grid, block, 0, s, a, cols, blocks, per);
    }
    hipLaunchKernelGGL((seq_conv_sum_kernel<K>), dim3((unsigned)((a.c + 31) / 32), a.dbias ? K + 1 : K), dim3(1024), 0, s,
                       a.work, parts, a.c, a.dw, a.dbias);
    return hipGetLastError();
  });
}

// V channels a lane where every buffer allows it, else one.
template <typename T, int V>
hipError_t run_wide(const ConvArgs& a, hipStream_t s) {
  constexpr int e = sizeof(T), bytes = V * e;
  const uintptr_t at = (uintptr_t)a.dx | (uintptr_t)a.state | (uintptr_t)a.dstate | (uintptr_t)a.dstate_out |
                       (uintptr_t)a.kept.e * e;
  const bool wide = a.c % V == 0 && pieces(a.dy, bytes, e) && (a.kept.q || pieces(a.x, bytes, e)) && at % bytes == 0;
  return wide ? run<T, V>(a, s) : run<T, 1>(a, s);
}

}  // namespace

}  // namespace convseq
