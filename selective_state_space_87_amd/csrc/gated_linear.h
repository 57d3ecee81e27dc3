// Device arithmetic of the gated linear recurrence (gfx950): what one element's
// inputs make of the state, and the derivatives.
//
//   u = gate + gate_bias;  g = u, softplus(u) or sigmoid(u);  a = e^(A g)
//   w = 1, sqrt(1 - a^2) or 1 - a;  v = x sigmoid(input_gate + input_bias) (or x)
//   h <- a h + w v
#pragma once

#include <hip/hip_runtime.h>

#include "device_math.h"
#include "gated_delta.h"
#include "gated_linear_args.h"

namespace ssm {

// 1 - e^la, given a = e^la. Near 0 the difference would cancel: the Taylor series
// of (e^x - 1) / x to x^5 is taken up to |x| = 1/4 (the first dropped term,
// x^6 / 5040, is below 2^-24 there); beyond, 1 - a is off by 2^-24 / 0.22 at most.
__device__ __forceinline__ float one_minus_decay(float la, float a) {
  const float s = fmaf(fmaf(fmaf(fmaf(fmaf(la, 1.0f / 720.0f, 1.0f / 120.0f), la, 1.0f / 24.0f), la, 1.0f / 6.0f), la,
                            0.5f), la, 1.0f);
  return fabsf(la) < 0.25f ? -la * s : 1.0f - a;
}

// sigmoid(u) and its derivative sigmoid(u) sigmoid(-u), from one exponential.
// (s (1 - s) would lose what is left of the derivative where s is near 1.)
__device__ __forceinline__ float sigmoid_slope(float u, float* slope) {
  const float v = exp_minus_abs(u), r = rcp_hw(1.0f + v);
  *slope = v * r * r;
  return u < 0.0f ? v * r : r;
}

template <int ACT>
__device__ __forceinline__ float gate_value(float u) {
  if constexpr (ACT == kGateSoftplus) {
    return gdr_softplus(u);
  } else if constexpr (ACT == kGateSigmoid) {
    return sigmoid_f(u);
  } else {
    return u;
  }
}

// The same with the gate's derivative.
template <int ACT>
__device__ __forceinline__ float gate_value_slope(float u, float* slope) {
  if constexpr (ACT == kGateSoftplus) {
    const float v = exp_minus_abs(u), w = 1.0f + v, r = rcp_hw(w);
    *slope = u < 0.0f ? v * r : r;
    return fmaxf(u, 0.0f) + fmaf(log2_hw(w), kLn2, v - (w - 1.0f));
  } else if constexpr (ACT == kGateSigmoid) {
    return sigmoid_slope(u, slope);
  } else {
    *slope = 1.0f;
    return u;
  }
}

__device__ __forceinline__ float decay(float la) { return exp2_hw(la * kLog2e); }

template <int SCALE>
__device__ __forceinline__ float input_weight(float la, float a) {
  if constexpr (SCALE == kInputNorm) {
    return __builtin_amdgcn_sqrtf(one_minus_decay(la, a) * (1.0f + a));  // 1 - a^2
  } else if constexpr (SCALE == kInputComplement) {
    return one_minus_decay(la, a);
  } else {
    return 1.0f;
  }
}

// dw / d la. Where a is 1 the square root has no derivative: 0 is taken.
template <int SCALE>
__device__ __forceinline__ float input_weight_slope(float a, float w) {
  if constexpr (SCALE == kInputNorm) {
    return w != 0.0f ? -a * a / w : 0.0f;
  } else if constexpr (SCALE == kInputComplement) {
    return -a;
  } else {
    return 0.0f;
  }
}

}  // namespace ssm
