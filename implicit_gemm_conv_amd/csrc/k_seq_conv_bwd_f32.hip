// k_seq_conv_bwd_f32.hip -- the backward kernels of seq_conv_bwd.h for float.
#include "seq_conv_bwd.h"

namespace convseq {

// Groups of 16 rows a wave walks.  Longer walks read fewer rows twice and leave
// fewer partial sums; shorter ones make more waves.  A wave's channels are
// taken as 128 whatever the type.  4 taps, bias, silu, 2048 channels, bf16, calls back to
// back in a graph on inputs in turn, with their sums, us at walks of 1, 2 and 4:
//   groups   from x                  from 8 bits
//   32768    104.5   94.0   93.8     119.3   95.0   86.6
//   16384     55.3   49.0   47.1      61.7   51.1   45.0
//    8192     31.9   28.1   28.8      33.1   27.7   29.0
//    4096     19.8   18.8   22.0      19.9   19.5   22.8
//    2048     13.7   14.3   19.0      14.5   15.4   21.7
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
