// seq_params.h -- plain parameter structs and launchers shared by the host
// side of include/convseq.h (seq_api.cpp) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convseq {

constexpr int kGroup = 16;  // rows of a channel that share a power of two in 8 bits
constexpr int kEvery = 64;  // rows between the recurrence's kept states
constexpr int kMaxTaps = 8;

// A (B, T, C) tensor with channel stride 1; strides in elements.
struct Rows {
  const void* p;
  int64_t sb, st;
};

// A (B, T, C) tensor in 8 bits: q (B, groups, 2, C, 8), e (B, groups, C).
struct Kept {
  int8_t* q;
  uint8_t* e;
};

// Whether every row of a view can be read in pieces of `bytes`, `elem` bytes an element.
inline bool pieces(const Rows& r, int bytes, int elem) {
  return ((uintptr_t)r.p | (uint64_t)(r.sb * elem) | (uint64_t)(r.st * elem)) % bytes == 0;
}

struct ConvArgs {
  int b, t, c, k, act, dtype;
  Rows x;
  Kept kept;  // forward: written if q; backward: read in place of x if q
  const void *w, *bias, *state;
  const uint8_t* starts;
  // forward
  void *y, *state_out;
  // backward
  Rows dy;
  const void* dstate_out;
  void *dx, *dstate;
  float *dw, *dbias, *work;
};

struct ConvStepArgs {
  int b, c, k, act, dtype, n_slots;
  const void* x;
  int64_t x_row;
  const void *w, *bias, *state;
  void* state_out;
  const int32_t* slots;
  void* y;
};

struct ScanArgs {
  int b, t, c, dtype;
  float decay;
  Rows x, r, i;
  Kept kept[3];
  const float *lam, *h0;
  const uint8_t* starts;
  // forward
  void* y;
  float *h_last, *states;
  // backward
  Rows dy;
  const float *states_in, *dh_last;
  void *dx, *dr, *di;
  float *dlam, *dh0;
  float* parts;  // the tiles' sums, in the workspace
  void* work;
};

struct ScanStepArgs {
  int b, c, dtype, n_slots;
  float decay;
  const void *x, *r, *i;
  int64_t x_row, r_row, i_row;
  const float *lam, *state;
  float* state_out;
  const int32_t* slots;
  void* y;
};

int conv_bwd_groups(int b, int t, int c);  // groups of 16 rows a wave of the backward pass walks
int conv_bwd_blocks(int t, int per);       // its workgroups along a sequence
int64_t conv_bwd_work_bytes(int b, int t, int c, int k);
int64_t scan_fwd_work_bytes(int b, int t, int c);
int64_t scan_bwd_work_bytes(int b, int t, int c);

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_bwd_f32(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_bwd_f16(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_bwd_bf16(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t s);
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_step(const ScanStepArgs& a, hipStream_t s);
hipError_t launch_pack8(int b, int t, int c, int dtype, const Rows& x, const Kept& kept, hipStream_t s);
hipError_t launch_unpack8(int b, int t, int c, int dtype, const Kept& kept, void* out, hipStream_t s);

}  // namespace convseq
