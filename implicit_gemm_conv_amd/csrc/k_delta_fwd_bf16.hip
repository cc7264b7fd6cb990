// k_delta_fwd_bf16.hip -- gated delta rule forward, bf16 (delta_fwd.h).
#include "delta_fwd.h"

namespace convdelta {

hipError_t launch_delta_fwd_bf16(const DeltaArgs& a, hipStream_t s) { return delta_fwd_of<__bf16>(a, s); }

}  // namespace convdelta
