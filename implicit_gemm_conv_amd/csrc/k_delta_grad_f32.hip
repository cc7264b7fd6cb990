// k_delta_grad_f32.hip -- gated delta rule, the gradients that add over all columns, f32 (delta_grad.h).
#include "delta_grad.h"

namespace convdelta {

hipError_t launch_delta_grad_f32(const DeltaArgs& a, hipStream_t s) { return delta_grad_of<float>(a, s); }

}  // namespace convdelta
