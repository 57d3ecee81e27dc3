// Interface between the C-ABI front end (api.cpp) and the RMS norm's launchers.
// Host-only types; nothing here crosses the public ABI.
#pragma once

#include <stdint.h>

namespace ssm {

struct RmsNormArgs {
  const void* x;
  const void* residual;   // or null
  const float* weight;    // or null
  void* y;
  void* residual_out;     // or null
  float* scales;          // or null
  int64_t rows, dim;
  int in_bf16, res_bf16, out_type;  // out_type: 0 float32, 1 bfloat16, 2 e4m3
  float eps;
};

struct RmsNormBwdArgs {
  const void* s;
  const float* weight;    // or null
  const float* dy;
  const float* dresidual; // or null
  float* ds;
  float* dweight;         // or null
  void* workspace;
  int64_t rows, dim;
  int s_bf16;
  float eps;
};

constexpr int64_t kRmsMaxDim = 16384;

// Weak: the validation front end also links without these kernels (a host-only
// build); a call that passes validation there reports a launch failure.
__attribute__((weak)) int launch_rms_norm(const RmsNormArgs& a, void* stream);
__attribute__((weak)) int launch_rms_norm_bwd(const RmsNormBwdArgs& a, void* stream);

// Blocks of the norm's backward, each with one partial row of dweight.
inline int64_t rms_norm_bwd_blocks(int64_t rows, int64_t dim) {
  const int64_t at_a_time = dim <= 1024 ? 4 : 1, groups = (rows + at_a_time - 1) / at_a_time;
  return groups < 512 ? groups : 512;
}

}  // namespace ssm
