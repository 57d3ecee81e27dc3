// Gated delta rule, the walk over a head's chunks: float32 inputs.
#include "gated_delta_chunk.h"

namespace ssm {

int launch_gdr_chunk_f(const GatedDeltaArgs& a, const GdrWork& ws, const GdrPlan& pl, bool backward, void* stream) {
  return gdr_launch_chunk<false>(a, ws, pl, backward, static_cast<hipStream_t>(stream));
}

}  // namespace ssm
