// Interface between the C-ABI front end (api.cpp) and the layer norm's and the
// dropout's launchers. Host-only types; nothing here crosses the public ABI.
#pragma once

#include <stdint.h>

namespace ssm {

// Dropout of an array: threshold 0 for none.
struct DropArgs {
  const int64_t* rng;   // {seed, step} on the device
  uint32_t call;
  uint32_t threshold;   // round(p 2^16), 0 .. 65536
  float scale;          // 65536 / (65536 - threshold); 0 where everything is dropped
};

inline DropArgs drop_args(const int64_t* rng, uint32_t call, double p) {
  const uint32_t t = static_cast<uint32_t>(p * 65536.0 + 0.5);
  return DropArgs{rng, call, t, t < 65536 ? static_cast<float>(65536.0 / (65536 - t)) : 0.0f};
}

struct LayerNormArgs {
  const void* x;
  const void* residual;   // or null
  const float* weight;    // or null
  const float* bias;      // or null
  void* y;
  void* residual_out;     // or null
  int64_t rows, dim;
  int in_bf16, res_bf16, out_bf16;
  float eps;
  DropArgs drop;          // of x
};

struct LayerNormBwdArgs {
  const void* s;
  const float* weight;    // or null
  const float* dy;
  const float* dresidual; // or null
  float* ds;
  float* dx;              // ds through the dropout, or null
  float* dweight;         // or null
  float* dbias;           // or null
  void* workspace;
  int64_t rows, dim;
  int s_bf16;
  float eps;
  DropArgs drop;
};

struct DropoutArgs {
  const void* x;
  const void* residual;   // or null
  void* y;
  int64_t n;
  int in_bf16, out_bf16;  // of x; of residual and y
  DropArgs drop;
};

constexpr int64_t kLayerNormMaxDim = 16384;

// Weak: the validation front end also links without these kernels (a host-only
// build); a call that passes validation there reports a launch failure.
__attribute__((weak)) int launch_layer_norm(const LayerNormArgs& a, void* stream);
__attribute__((weak)) int launch_layer_norm_bwd(const LayerNormBwdArgs& a, void* stream);
__attribute__((weak)) int launch_dropout(const DropoutArgs& a, void* stream);

// Blocks of the norm's backward, each with one partial row of dweight and one
// of dbias. Rows up to 1024 elements go four to a block. Two blocks a CU. Calls with 512,
// 768, 1024 blocks, float32 (us): (32768, 4096) with a residual 402, 416, 419; (65536, 1024)
// 148, 168, 152; (1000, 1537) 16, 17, 20; (8192, 16384) 338, 358, 371; but (32768, 1536)
// 134, 112, 113, and of narrow rows, which are a turn's latency after another, 10^6 of 64
// 776, 551, 454 and 10^6 of 128 817, 588, 478.
inline int64_t layer_norm_bwd_blocks(int64_t rows, int64_t dim) {
  const int64_t at_a_time = dim <= 1024 ? 4 : 1, groups = (rows + at_a_time - 1) / at_a_time;
  return groups < 512 ? groups : 512;
}

// Turns of a block (a row each, or four) after which its sums go to second ones.
constexpr int64_t kLayerNormFold = 64;

}  // namespace ssm
