// k_delta_grad_bf16.hip -- gated delta rule, the gradients that add over all columns, bf16 (delta_grad.h).
#include "delta_grad.h"

namespace convdelta {

hipError_t launch_delta_grad_bf16(const DeltaArgs& a, hipStream_t s) { return delta_grad_of<__bf16>(a, s); }

}  // namespace convdelta
