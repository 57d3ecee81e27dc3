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

// The exponents are taken in base 2 and the parameters come scaled: A2 = A log2(e),
// and for a sigmoid the bias as -bias log2(e), so that its exponent is one fused
// product and sum. That exponent's rounding, and the bias's, are 2^-24 (|u| + |bias|) of
// e^-u, and so of a gate far down the sigmoid. A compensated exponent takes four
// instructions more a gate, eight on the 37 an element that the forward has, which
// fill 0.6 of its time: they are left out.

// 1 - 2^t for t <= 0, given a = 2^t. Near 0 the difference would cancel: the Taylor
// series of (e^x - 1) / x to x^5, x = t ln 2, is taken up to |x| = 1/4 (the first
// dropped term, x^6 / 5040, is below 2^-24 there); beyond, `far` is off by some
// 2^-24 / 0.22.
__device__ __forceinline__ float one_minus_exp2(float t, float far) {
  constexpr float l = kLn2, l2 = l * l, l3 = l2 * l, l4 = l3 * l, l5 = l4 * l, l6 = l5 * l;
  const float s = fmaf(fmaf(fmaf(fmaf(fmaf(t, -l6 / 720.0f, -l5 / 120.0f), t, -l4 / 24.0f), t, -l3 / 6.0f), t,
                            -l2 / 2.0f), t, -l);
  return fabsf(t) < 0.25f * kLog2e ? t * s : far;
}

// sigmoid(x + bias), given -bias log2(e). (e is infinite below -88: 0.)
__device__ __forceinline__ float glr_sigmoid(float x, float nb) { return rcp_hw(1.0f + exp2_hw(fmaf(x, -kLog2e, nb))); }

// The same with its derivative s (1 - s) = e s^2, which keeps what is left of it
// where s is near 1. (The exponent ends at 126: 0 times infinity would be NaN.)
__device__ __forceinline__ float glr_sigmoid_slope(float x, float nb, float* slope) {
  float t = fmaf(x, -kLog2e, nb);
  t = t > 126.0f ? 126.0f : t;
  const float e = exp2_hw(t), r = rcp_hw(1.0f + e);
  *slope = e * r * r;
  return r;
}

// max(u, 0) + log1p(v), v = e^-|u|, as in softplus_f; the slope is sigmoid(u).
__device__ __forceinline__ float glr_softplus(float u, float* slope) {
  const float v = exp2_hw(-fabsf(u) * kLog2e), w = 1.0f + v;
  if (slope != nullptr) *slope = (u < 0.0f ? v : 1.0f) * rcp_hw(w);
  return fmaxf(u, 0.0f) + fmaf(log2_hw(w), kLn2, v - (w - 1.0f));
}

// Value of the gate (and its derivative) given its raw value and the scaled bias.
template <int ACT>
__device__ __forceinline__ float gate_value(float x, float bias) {
  if constexpr (ACT == kGateSoftplus) {
    return glr_softplus(x + bias, nullptr);
  } else if constexpr (ACT == kGateSigmoid) {
    return glr_sigmoid(x, bias);
  } else {
    return x + bias;
  }
}
template <int ACT>
__device__ __forceinline__ float gate_value_slope(float x, float bias, float* slope) {
  if constexpr (ACT == kGateSoftplus) {
    return glr_softplus(x + bias, slope);
  } else if constexpr (ACT == kGateSigmoid) {
    return glr_sigmoid_slope(x, bias, slope);
  } else {
    *slope = 1.0f;
    return x + bias;
  }
}

// Weight of the input, given t = log2(a) and a. sqrt(1 - a^2): 1 - 2^(2t).
template <int SCALE>
__device__ __forceinline__ float input_weight(float t, float a) {
  if constexpr (SCALE == kInputNorm) {
    return __builtin_amdgcn_sqrtf(one_minus_exp2(2.0f * t, fmaf(-a, a, 1.0f)));
  } else if constexpr (SCALE == kInputComplement) {
    return one_minus_exp2(t, 1.0f - a);
  } else {
    return 1.0f;
  }
}

// dw / d(ln a). Where a is 1 the square root has no derivative: 0 is taken.
template <int SCALE>
__device__ __forceinline__ float input_weight_slope(float a, float w) {
  if constexpr (SCALE == kInputNorm) {
    return w != 0.0f ? -a * a * rcp_hw(w) : 0.0f;
  } else if constexpr (SCALE == kInputComplement) {
    return -a;
  } else {
    return 0.0f;
  }
}

}  // namespace ssm
