// Interface between the C-ABI front end (api.cpp) and the launcher of the causal
// convolution's gradients, and the plan of a call. Host-only types; nothing here
// crosses the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ssm {

struct ConvBwdArgs {
  const void* x;
  const float* weight;
  const float* bias;         // or null
  const float* state_in;     // or null
  const float* dy;
  const float* dstate_out;   // or null
  float* dx;
  float* dweight;            // or null
  float* dbias;              // or null
  float* dstate_in;          // or null
  void* workspace;
  int64_t batch, seqlen, dim, width;
  int in_bf16, silu;
};

// Weak: the validation front end also links without these kernels (a host-only
// build); a call that passes validation there reports a launch failure.
__attribute__((weak)) int launch_conv1d_bwd(const ConvBwdArgs& a, void* stream);

// A batch row's steps are walked in `segs` segments of `seg` steps at the same
// time; each leaves its part of the filters' gradients, [parts][width + 1][dim].
struct ConvBwdPlan {
  int64_t seg, segs;
  size_t bytes;
};

// As many segments as make kConvBwdWaves waves, 8 a CU: they are all there at once
// (12 would fit at width 4, and 8 at width 8), and their parts are few. Measured (the call)
// at (4, 8192, 4096, width 4): 8, 12, 16, 32 waves a CU 250, 280, 265, 266 us in bfloat16,
// 298, 331, 345, 341 in float32; (1, 4096, 2560) bfloat16 33, 37, 37, 36.
constexpr int64_t kConvBwdMinSeg = 16, kConvBwdMaxSeg = 512, kConvBwdWaves = 2048;

inline ConvBwdPlan plan_conv1d_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width) {
  ConvBwdPlan p{};
  const auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int64_t groups = batch * ceil_div(dim, 256);  // waves, of four channels a thread
  const int64_t wanted = ceil_div(kConvBwdWaves, groups > 0 ? groups : 1);
  int64_t seg = ceil_div(ceil_div(seqlen, wanted), 16) * 16;
  seg = seg < kConvBwdMinSeg ? kConvBwdMinSeg : (seg > kConvBwdMaxSeg ? kConvBwdMaxSeg : seg);
  p.seg = seg;
  p.segs = seqlen > 0 ? ceil_div(seqlen, seg) : 1;
  p.bytes = static_cast<size_t>(batch * p.segs) * static_cast<size_t>((width + 1) * dim) * 4;
  return p;
}

}  // namespace ssm
