// Forward tiles of the gated linear recurrence for bfloat16 inputs (see gated_linear_fwd.h).
#include "gated_linear_fwd.h"

namespace ssm {

template void launch_glr_fwd<true>(const GatedLinearArgs& a, const GlrChainPlan& plan, hipStream_t st);

}  // namespace ssm
