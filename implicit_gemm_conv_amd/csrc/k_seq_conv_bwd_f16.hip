// k_seq_conv_bwd_f16.hip -- the backward kernels of seq_conv_bwd.h for _Float16.
#include "seq_conv_bwd.h"

namespace convseq {

hipError_t launch_conv_bwd_f16(const ConvArgs& a, hipStream_t s) { return run_wide<_Float16, 2>(a, s); }

}  // namespace convseq
