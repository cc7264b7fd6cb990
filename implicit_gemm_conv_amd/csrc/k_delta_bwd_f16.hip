// k_delta_bwd_f16.hip -- gated delta rule, the backward recurrence, f16 (delta_bwd.h).
#include "delta_bwd.h"

namespace convdelta {

hipError_t launch_delta_bwd_f16(const DeltaArgs& a, hipStream_t s) { return delta_bwd_of<_Float16>(a, s); }

}  // namespace convdelta
