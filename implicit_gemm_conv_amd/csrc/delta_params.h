// delta_params.h -- plain parameter structs, workspace layout and launchers
// shared by the host side of include/convdelta.h (delta_api.cpp) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convdelta {

constexpr int kChunk = 64;  // rows taken at a time; rows between the kept states
constexpr int kMaxDk = 128;
constexpr int kFrag = 1024;               // bytes of one 16x32 operand of 16-bit parts
constexpr int kTri = 6;                   // 16x32 operands that cover a 64x64 triangle
constexpr int kParts = 3;                 // 16-bit parts that hold an fp32 value
constexpr int kMatrix = kTri * kParts * kFrag;

// A (B, T, H, D) tensor with element stride 1; strides in elements.
struct Heads {
  const void* p;
  int64_t sb, st, sh;
};

// What the preparing kernel leaves for each chunk of each head (index
// ((b * Hv + h) * chunks + c) throughout).
struct Work {
  char* solve;     // forward: H as operands of x = r + H (beta r), kMatrix bytes
  char* read;      // ... and the decayed q k^T, the same way
  char* solve_t;   // backward: the transposes of both
  char* read_t;
  float* rows;     // 4 x 64: enter, leave, beta, step (see delta_device.h)
  double* sums;    // backward: 64 sums of log decays
  int* seq;        // backward: 64 sequence numbers inside the chunk
  float* z;        // backward: z, (B * Hv, chunks * 64, dvp)
  float* dstate;   // backward: the gradient of the state after each chunk, (.., Dk, dvp)
  void *q, *k;     // (B, Hk, T, dkp) copies, where q or k are not 16-byte aligned rows of whole 16 bytes, or far apart
};

struct DeltaArgs {
  int b, t, hk, hv, dk, dv, dtype;
  int chunks, dvp;  // ceil(T / 64); Dv rounded up to 32
  int dkp;          // elements of a row of q and k as the kernels read them: Dk rounded up to 8
  int whole;        // dy's rows are whole pieces of 8 elements, 16-byte aligned
  float scale;
  Heads q, k, v, dy;
  const float *log_decay, *beta, *h0, *states_in, *x_in, *dh_last;
  const uint8_t* starts;
  void *y, *dq, *dk_, *dv_;
  float *h_last, *states, *x, *dlog_decay, *dbeta, *dh0;
  Work w;
};

// Rows of one chunk c of one head of a dense (B, T, Hv, Dv) tensor: where they begin, and the bytes to the end of the last
// row's own Dv, both in bytes.  (The rest of that row, other heads, may be past the tensor's end.)
struct Span {
  int64_t at, bytes;
};
inline __host__ __device__ Span dense_rows(const DeltaArgs& a, int b, int h, int c, int elem) {
  const int left = a.t - c * kChunk, rows = left < kChunk ? left : kChunk;
  const int64_t row = (int64_t)a.hv * a.dv;
  return {(((int64_t)b * a.t + c * kChunk) * row + (int64_t)h * a.dv) * elem, ((rows - 1) * row + a.dv) * elem};
}

// Those copies: a head's rows one after the other, so that 64 of them have offsets of 32 bits however many heads there are.
inline __host__ __device__ Heads packed_rows(const void* p, int t, int hk, int dkp) {
  return {p, (int64_t)hk * t * dkp, dkp, (int64_t)t * dkp};
}

struct DeltaStepArgs {
  int b, hk, hv, dk, dv, dtype, n_slots;
  float scale;
  Heads q, k, v;
  const float *log_decay, *beta, *state;
  float* state_out;
  const int32_t* slots;
  void* y;
};

hipError_t launch_delta_pack(const DeltaArgs& a, const Heads& q, const Heads& k, hipStream_t s);
hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t s);
// One launcher for each type:
//   fwd     y, the states
//   bwd     dv, z, the states' gradients
//   grad    dq, dk, dlog_decay, dbeta
#define CONVDELTA_LAUNCHERS(type)                                        \
  hipError_t launch_delta_fwd_##type(const DeltaArgs& a, hipStream_t s);    \
  hipError_t launch_delta_bwd_##type(const DeltaArgs& a, hipStream_t s);    \
  hipError_t launch_delta_grad_##type(const DeltaArgs& a, hipStream_t s);
CONVDELTA_LAUNCHERS(f32)
CONVDELTA_LAUNCHERS(f16)
CONVDELTA_LAUNCHERS(bf16)
#undef CONVDELTA_LAUNCHERS
hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s);

}  // namespace convdelta
