// delta_team.h -- what the forward and the backward recurrence of the gated delta
// rule share: where a lane of the eight waves stands, the columns of parts in LDS, and
// the operands that a wave fetches for a chunk.
#pragma once

#include "delta_device.h"

namespace convdelta {

constexpr int kTeam = 512;  // two roles of four waves

// Columns of parts: [part][16 columns][ld].  The 8 spare elements spread the columns over the banks.
template <int LEN>
struct ColsAt {
  static constexpr int ld = LEN + 8, part = 16 * ld;
};

// A workgroup's columns: NC tiles of 16.
template <typename T, int DK, int NC>
struct Team {
  static constexpr int NP = InParts<T>::n, KS = DK / 32, DT = DK / 16;
  typedef ColsAt<DK> State;
  typedef ColsAt<kChunk> Rows;

  const DeltaArgs& a;
  int wave, tile, m, q4, lane, b, h, hk, bh, block;  // tile: the wave's 16 rows of the state, where it is below DT

  __device__ __forceinline__ Team(const DeltaArgs& a_, int bh_, int cb) : a(a_), bh(bh_), block(cb * 16 * NC) {
    lane = threadIdx.x % 64;
    wave = wave_id() % 4;
    // the second role has less to do before the state: with few tiles it takes them
    tile = DT == 8 ? wave_id() : wave_id() - 4;
    m = lane % 16;
    q4 = lane / 16;
    b = bh / a.hv;
    h = bh % a.hv;
    hk = h / (a.hv / a.hk);
  }
  __device__ __forceinline__ int col(int n) const { return block + 16 * n + m; }  // the lane's column of tile n
  __device__ __forceinline__ int row() const { return 16 * wave + 4 * q4; }  // the first of the lane's four
  __device__ __forceinline__ bool has_tile() const { return tile >= 0 && tile < DT; }

  // the lane's 4 values a tile of a (Dk, Dv) state, zero outside
  __device__ __forceinline__ void load_state(const float* from, f32x4_t (&s)[NC]) const {
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 16 * tile + 4 * q4 + r;
        s[n][r] = from && col(n) < a.dv && has_tile() && d < a.dk ? from[(int64_t)d * a.dv + col(n)] : 0.f;
      }
  }
  // ... into a (Dk, ld) state of which the columns below `width` are there; nowhere if `to` is NULL
  __device__ __forceinline__ void store_state(float* to, int ld, int width, const f32x4_t (&s)[NC]) const {
    const Range x(to, to ? (int64_t)a.dk * ld * 4 : 0);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const uint32_t at = col(n) < width && has_tile() ? (uint32_t)((16 * tile + 4 * q4) * ld + col(n)) * 4u : kNowhere;
#pragma unroll
      for (int r = 0; r < 4; ++r) x.store(at + (uint32_t)(r * ld) * 4u, s[n][r]);
    }
  }
  // four neighbouring rows of the lane's column, as parts
  template <int N, typename AT>
  __device__ __forceinline__ void put(__bf16* cols, int at, const f32x4_t& x) const {
    bf164_t o[N];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      __bf16 w[N];
      split_one<N>(x[r], w);
#pragma unroll
      for (int n = 0; n < N; ++n) o[n][r] = w[n];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) *(bf164_t*)(cols + n * AT::part + m * AT::ld + at) = o[n];
  }
  __device__ __forceinline__ void put_state(__bf16 (&cols)[NC][kParts * State::part], const f32x4_t (&s)[NC]) const {
    if (!has_tile()) return;
#pragma unroll
    for (int n = 0; n < NC; ++n) put<kParts, State>(cols[n], 16 * tile + 4 * q4, s[n]);
  }
  // the operand of step k of a contraction over the state's rows, or over the chunk's
  template <int N, typename AT>
  __device__ __forceinline__ Parts<N> get(const __bf16* cols, int k) const {
    return natural<N>(cols + m * AT::ld + 32 * k + 8 * q4, AT::part);
  }
  // columns of state tile t of a chunk's rows in LDS, as rows; step k over the chunk's rows
  __device__ __forceinline__ Parts<NP> cols_of(const __bf16* x, int t, int k) const {
    return transposed<NP>(x + (32 * k + 8 * q4 + m / 4) * RowsAt<DK>::stride + 16 * t + 4 * (m % 4), RowsAt<DK>::stride,
                          RowsAt<DK>::part);
  }
  // this wave's rows of q or k
  __device__ __forceinline__ void load_rows(const Heads& x, int c, Raw8<T> (&to)[KS]) const {
    const Range p = rows_range<T>(x, b, hk, c * kChunk, a.t, a.dkp);
#pragma unroll
    for (int k = 0; k < KS; ++k) to[k].load(p, (16 * wave + m) * row_bytes<T>(x), 32 * k + 8 * q4, a.dkp);
  }
  __device__ __forceinline__ Parts<NP> rows_of(const Raw8<T> (&x)[KS], int k) const { return x[k].parts(); }
  // ... into LDS, row by row
  __device__ __forceinline__ void put_rows(__bf16* to, const Raw8<T> (&x)[KS]) const {
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const Parts<NP> p = rows_of(x, k);
#pragma unroll
      for (int n = 0; n < NP; ++n) *(bf168_t*)(to + n * RowsAt<DK>::part + (16 * wave + m) * RowsAt<DK>::stride + 32 * k + 8 * q4) = p.p[n];
    }
  }
  // the lane's four rows of its columns of v or of y's gradient; zero past Dv (and past T, if rows do not overlap)
  __device__ __forceinline__ void load_col(const Heads& x, int c, T (&to)[NC][4]) const {
    const Range p = rows_range<T>(x, b, h, c * kChunk, a.t, a.dv);
    const uint32_t ld = row_bytes<T>(x);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const uint32_t at = col(n) < a.dv ? row() * ld + (uint32_t)col(n) * (uint32_t)sizeof(T) : kNowhere;
#pragma unroll
      for (int r = 0; r < 4; ++r) to[n][r] = p.load<T>(at + r * ld);
    }
  }
  // ... and of y, x or v's gradient, dense, rows past T left out
  template <typename E>
  __device__ __forceinline__ void store_col(void* to, int c, const f32x4_t (&v)[NC], int first = 0, int end = kChunk) const {
    const uint32_t ld = (uint32_t)(a.hv * a.dv) * (uint32_t)sizeof(E);
    const Span rows = dense_rows(a, b, h, c, sizeof(E));
    const Range p((char*)to + rows.at, rows.bytes);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const uint32_t at = col(n) < a.dv ? row() * ld + (uint32_t)col(n) * (uint32_t)sizeof(E) : kNowhere;
#pragma unroll
      for (int r = 0; r < 4; ++r) p.store(row() + r >= first && row() + r < end ? at + r * ld : kNowhere, from_f32<E>(v[n][r]));
    }
  }
  __device__ __forceinline__ f32x4_t load_gate(int which, int c) const {
    return load_at<f32x4_t>(a.w.rows + (chunk_index(a, bh, c) * 4 + which) * kChunk, 4u * row());
  }
  // the last row's enter
  __device__ __forceinline__ float load_stay(int c) const {
    return load_at<float>(a.w.rows + chunk_index(a, bh, c) * 4 * kChunk, 4u * (kChunk - 1));
  }
  // this wave's operands of a triangular matrix: of a lower one steps 0 and, from wave 2 on, 1; of an
  // upper one (UP) step 1 and, up to wave 1, 0
  template <bool UP>
  __device__ __forceinline__ bool has(int k) const { return UP ? k >= wave / 2 : k <= wave / 2; }
  template <bool UP, int N>
  __device__ __forceinline__ void load_matrix(const char* x, int c, Parts<N> (&to)[2]) const {
    const char* p = x + chunk_index(a, bh, c) * kMatrix;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // the operand's number in the order of low_t, low_s (up_t, up_s); one that is not there repeats the other
      const int f = UP ? (wave < 2 ? 2 * wave + k : wave + 2) : (wave < 2 ? wave : 2 * wave - 2 + k);
#pragma unroll
      for (int n = 0; n < N; ++n) to[k].p[n] = load_at<bf168_t>(p + f * kParts * kFrag, n * kFrag + lane * 16u);
    }
  }
};

}  // namespace convdelta
