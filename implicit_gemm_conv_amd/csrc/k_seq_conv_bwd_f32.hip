// k_seq_conv_bwd_f32.hip -- the backward kernels of seq_conv_bwd.h for float.
#include "seq_conv_bwd.h"

namespace convseq {

// Groups of 16 rows a wave walks.  Longer walks read fewer rows twice and leave
// fewer partial sums; shorter ones make more waves.  A wave's channels are
// taken as 128 whatever the type.  4 taps, silu, bf16, backward with its sums, at
// 1, 2 and 4 groups: 16384 groups (4x4096x2048) 52.3, 45.6 and 41.0 us; 8192 30.7,
// 26.0 and 27.3; 4096 18.7, 18.4 and 20.9; 2048 13.3, 14.4 and 19.0.
int conv_bwd_groups(int b, int t, int c) {
  const int64_t groups = (int64_t)b * ((t + kGroup - 1) / kGroup) * ((c + 127) / 128);
  return groups >= 16384 ? 4 : groups >= 8192 ? 2 : 1;
}
int conv_bwd_blocks(int t, int per) {
  const int rows = per * kGroup * kWaves;
  return t > 0 ? (t + rows - 1) / rows : 1;
}
int64_t conv_bwd_work_bytes(int b, int t, int c, int k) {
  return (int64_t)b * conv_bwd_blocks(t, conv_bwd_groups(b, t, c)) * (k + 1) * c * 4;
}

hipError_t launch_conv_bwd_f32(const ConvArgs& a, hipStream_t s) { return run<float, 1>(a, s); }

}  // namespace convseq
