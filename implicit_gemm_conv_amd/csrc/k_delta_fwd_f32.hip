// k_delta_fwd_f32.hip -- gated delta rule forward, f32 (delta_fwd.h).
#include "delta_fwd.h"

namespace convdelta {

hipError_t launch_delta_fwd_f32(const DeltaArgs& a, hipStream_t s) { return delta_fwd_of<float>(a, s); }

}  // namespace convdelta
