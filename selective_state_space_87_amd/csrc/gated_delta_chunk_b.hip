// Gated delta rule, the walk over a head's chunks: bfloat16 inputs.
#include "gated_delta_chunk.h"

namespace ssm {

int launch_gdr_chunk_b(const GatedDeltaArgs& a, const GdrWork& ws, const GdrPlan& pl, bool backward, void* stream) {
  return gdr_launch_chunk<true>(a, ws, pl, backward, static_cast<hipStream_t>(stream));
}

}  // namespace ssm
