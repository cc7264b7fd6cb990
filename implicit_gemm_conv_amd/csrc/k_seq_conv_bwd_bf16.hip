// k_seq_conv_bwd_bf16.hip -- the backward kernels of seq_conv_bwd.h for __bf16.
#include "seq_conv_bwd.h"

namespace convseq {

hipError_t launch_conv_bwd_bf16(const ConvArgs& a, hipStream_t s) { return run_wide<__bf16, 2>(a, s); }

}  // namespace convseq
