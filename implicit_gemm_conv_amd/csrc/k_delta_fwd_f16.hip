// k_delta_fwd_f16.hip -- gated delta rule forward, f16 (delta_fwd.h).
#include "delta_fwd.h"

namespace convdelta {

hipError_t launch_delta_fwd_f16(const DeltaArgs& a, hipStream_t s) { return delta_fwd_of<_Float16>(a, s); }

}  // namespace convdelta
