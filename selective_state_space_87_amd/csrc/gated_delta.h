// Device helpers shared by the gated delta rule's kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include "device_math.h"
#include "gated_delta_args.h"

namespace ssm {

// Steps of a batch row: its entry of seqlens, within [0, L].
__device__ __forceinline__ int64_t gdr_row_steps(const int32_t* seqlens, int b, int64_t L) {
  if (seqlens == nullptr) return L;
  const int64_t n = seqlens[b];
  return n < 0 ? 0 : (n > L ? L : n);
}

// Step size and log decay dt A of one step. A log decay below -200 becomes
// -200 (its exponential is 0 in float32 either way), so that sums of log
// decays stay finite; NaN stays NaN.
__device__ __forceinline__ float gdr_step(const GatedDeltaArgs& p, float raw, float bias) {
  const float x = raw + bias;
  return p.dt_softplus ? softplus_f(x) : x;
}
__device__ __forceinline__ float gdr_clamp_decay(float g) { return g < kGdrMinLogDecay ? kGdrMinLogDecay : g; }
__device__ __forceinline__ float gdr_log_decay(const GatedDeltaArgs& p, float raw, float bias, float A) {
  return gdr_clamp_decay(gdr_step(p, raw, bias) * A);
}

__device__ __forceinline__ float sigmoid_f(float x) { return rcp_hw(1.0f + exp2_hw(-x * kLog2e)); }
__device__ __forceinline__ float gdr_beta(const GatedDeltaArgs& p, float raw) {
  return p.beta_sigmoid ? sigmoid_f(raw) : raw;
}

}  // namespace ssm
