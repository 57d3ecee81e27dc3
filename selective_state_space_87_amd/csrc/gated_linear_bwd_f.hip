// Backward tiles of the gated linear recurrence for float32 inputs (see gated_linear_bwd.h).
#include "gated_linear_bwd.h"

namespace ssm {

template void launch_glr_bwd<false>(const GatedLinearBwdArgs& a, const GlrBwdPlan& plan, hipStream_t st);

}  // namespace ssm
