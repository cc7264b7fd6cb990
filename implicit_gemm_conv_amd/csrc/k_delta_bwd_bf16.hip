// k_delta_bwd_bf16.hip -- gated delta rule, the backward recurrence, bf16 (delta_bwd.h).
#include "delta_bwd.h"

namespace convdelta {

hipError_t launch_delta_bwd_bf16(const DeltaArgs& a, hipStream_t s) { return delta_bwd_of<__bf16>(a, s); }

}  // namespace convdelta
