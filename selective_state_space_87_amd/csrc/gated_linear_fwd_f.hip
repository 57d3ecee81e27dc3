// Forward tiles of the gated linear recurrence for float32 inputs (see gated_linear_fwd.h).
#include "gated_linear_fwd.h"

namespace ssm {

template void launch_glr_fwd<false>(const GatedLinearArgs& a, const GlrChainPlan& plan, hipStream_t st);

}  // namespace ssm
