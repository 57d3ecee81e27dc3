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

// e^-|x|: the exponent in base 2 with what its rounding, and log2(e)'s, left out
// (|x| 2^-24 and |x| 2^-26, the same way at every step: 1e-7 of a step size at x = -6).
__device__ __forceinline__ float exp_minus_abs(float x) {
  constexpr float kLog2eLo = 1.92596299e-8f;  // log2(e) - kLog2e
  const float y = -fabsf(x), t = y * kLog2e, e = exp2_hw(t);
  const float left = fmaf(y, kLog2eLo, fmaf(y, kLog2e, -t));
  return y < -126.0f ? 0.0f : fmaf(e, left * kLn2, e);  // (infinity would leave NaN; e is 0 from -104 on)
}
__device__ __forceinline__ float sigmoid_f(float x) {
  const float v = exp_minus_abs(x);
  return (x < 0.0f ? v : 1.0f) * rcp_hw(1.0f + v);
}
// max(x, 0) + log1p(v), v = e^-|x| (see softplus_f).
__device__ __forceinline__ float gdr_softplus(float x) {
  const float v = exp_minus_abs(x), w = 1.0f + v;
  return fmaxf(x, 0.0f) + fmaf(log2_hw(w), kLn2, v - (w - 1.0f));
}

// Step size and log decay dt A of one step. A log decay below -200 becomes
// -200 (its exponential is 0 in float32 either way), so that sums of log
// decays stay finite; NaN stays NaN.
__device__ __forceinline__ float gdr_step(const GatedDeltaArgs& p, float raw, float bias) {
  const float x = raw + bias;
  return p.dt_softplus ? gdr_softplus(x) : x;
}
__device__ __forceinline__ float gdr_clamp_decay(float g) { return g < kGdrMinLogDecay ? kGdrMinLogDecay : g; }
__device__ __forceinline__ float gdr_log_decay(const GatedDeltaArgs& p, float raw, float bias, float A) {
  return gdr_clamp_decay(gdr_step(p, raw, bias) * A);
}

__device__ __forceinline__ float gdr_beta(const GatedDeltaArgs& p, float raw) {
  return p.beta_sigmoid ? sigmoid_f(raw) : raw;
}

}  // namespace ssm
