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

// The decay's exponent is taken in base 2 and its parameter comes scaled: A2 = A log2(e).
//
// A gate's exponential e^y, y = -u or -|u|, is compensated: with t = y log2(e), rounded,
// e^y = 2^t e^(y - t ln 2), and what is left, y - t ln 2, is one fused product and sum
// (ln 2's own rounding is 0.05 2^-24 |y| of it) and at most 1.3 2^-24 |y|, so that e^y is
// 2^t q with q = 1 + y - t ln 2. Without q a gate far down the sigmoid would be off by that
// much beside what the sum u was rounded by. It takes five instructions more a gate, 45
// for 37 an element with both, which the loads hide (the call at (4, 8192, 4096) bfloat16
// 214 us for 214; 64 rows of 128 steps, one tile each, 64 for 62); e^-|u| as gated_delta.h
// takes it costs ten (238).
struct GlrExp {
  float e, q;  // 2^t and q: the product is left to what takes it
};
__device__ __forceinline__ GlrExp glr_exp(float y, float t) { return GlrExp{exp2_hw(t), 1.0f + fmaf(t, -kLn2, y)}; }

// 1 - 2^(TIMES t) for t <= 0. Near 0 the difference would cancel: the Taylor series of
// (e^x - 1) / x to x^5, x = TIMES t ln 2, is taken up to |x| = 1/4 (the first dropped term,
// x^6 / 5040, is below 2^-24 there); beyond, `far`, the difference itself, is off by some
// 2^-24 / 0.22.
template <int TIMES>
__device__ __forceinline__ float one_minus_exp2(float t, float far) {
  constexpr float l = TIMES * kLn2, l2 = l * l, l3 = l2 * l, l4 = l3 * l, l5 = l4 * l, l6 = l5 * l;
  const float s = fmaf(fmaf(fmaf(fmaf(fmaf(t, -l6 / 720.0f, -l5 / 120.0f), t, -l4 / 24.0f), t, -l3 / 6.0f), t,
                            -l2 / 2.0f), t, -l);
  return fabsf(t) < 0.25f / TIMES * kLog2e ? t * s : far;
}

// e^-u, of which the sigmoid is made: u ends at 88, where the sigmoid is 1 (infinity would
// leave NaN behind it), and t at 126, where it is 0: q then takes the value beyond
// float32 for u = -infinity. NaN stays, by the first minimum or in q.
__device__ __forceinline__ GlrExp glr_sigmoid_exp(float u) {
  u = __builtin_elementwise_minimum(u, 88.0f);
  return glr_exp(-u, fminf(u * -kLog2e, 126.0f));
}
__device__ __forceinline__ float glr_sigmoid(float u) {
  const GlrExp v = glr_sigmoid_exp(u);
  return rcp_hw(fmaf(v.e, v.q, 1.0f));
}
// The same with its derivative s (1 - s) = s (e^-u s), which keeps what is left of it
// where s is near 1. (Where s is 0, infinity times it: the minimum makes 1 of that.)
__device__ __forceinline__ float glr_sigmoid_slope(float u, float* slope) {
  const GlrExp v = glr_sigmoid_exp(u);
  const float s = rcp_hw(fmaf(v.e, v.q, 1.0f));
  *slope = s * fminf(v.e * v.q * s, 1.0f);
  return s;
}

// max(u, 0) + log1p(v), v = e^-|u|, as in softplus_f; the slope is sigmoid(u).
__device__ __forceinline__ float glr_softplus(float u, float* slope) {
  const float y = __builtin_elementwise_maximum(-fabsf(u), -126.0f);
  const GlrExp x = glr_exp(y, y * kLog2e);
  const float v = x.e * x.q, w = 1.0f + v;
  if (slope != nullptr) *slope = (u < 0.0f ? v : 1.0f) * rcp_hw(w);
  return fmaxf(u, 0.0f) + fmaf(log2_hw(w), kLn2, v - (w - 1.0f));
}

// Value of the gate (and its derivative).
template <int ACT>
__device__ __forceinline__ float gate_value(float u) {
  if constexpr (ACT == kGateSoftplus) {
    return glr_softplus(u, nullptr);
  } else if constexpr (ACT == kGateSigmoid) {
    return glr_sigmoid(u);
  } else {
    return u;
  }
}
template <int ACT>
__device__ __forceinline__ float gate_value_slope(float u, float* slope) {
  if constexpr (ACT == kGateSoftplus) {
    return glr_softplus(u, slope);
  } else if constexpr (ACT == kGateSigmoid) {
    return glr_sigmoid_slope(u, slope);
  } else {
    *slope = 1.0f;
    return u;
  }
}

// Weight of the input, given t = log2(a) and a. sqrt(1 - a^2): 1 - 2^(2t).
template <int SCALE>
__device__ __forceinline__ float input_weight(float t, float a) {
  if constexpr (SCALE == kInputNorm) {
    return __builtin_amdgcn_sqrtf(one_minus_exp2<2>(t, fmaf(-a, a, 1.0f)));
  } else if constexpr (SCALE == kInputComplement) {
    return one_minus_exp2<1>(t, 1.0f - a);
  } else {
    return 1.0f;
  }
}

// dw / d(ln a). Where a is 1 the square root has no derivative: 0 is taken. (The hardware's
// reciprocal is off by one unit in the last place, half a unit more than a division of
// ten instructions; w itself is off by several where 1 - a^2 cancels.)
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
