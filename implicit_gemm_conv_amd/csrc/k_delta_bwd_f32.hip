// k_delta_bwd_f32.hip -- gated delta rule, the backward recurrence, f32 (delta_bwd.h).
#include "delta_bwd.h"

namespace convdelta {

hipError_t launch_delta_bwd_f32(const DeltaArgs& a, hipStream_t s) { return delta_bwd_of<float>(a, s); }

}  // namespace convdelta
