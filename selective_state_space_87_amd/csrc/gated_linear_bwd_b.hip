// Backward tiles of the gated linear recurrence for bfloat16 inputs (see gated_linear_bwd.h).
#include "gated_linear_bwd.h"

namespace ssm {

template void launch_glr_bwd<true>(const GatedLinearBwdArgs& a, const GlrBwdPlan& plan, hipStream_t st);

}  // namespace ssm
