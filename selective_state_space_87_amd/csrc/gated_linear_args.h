// Interface between the C-ABI front end (api.cpp) and the gated linear
// recurrence's launchers, and the plan of a call. Host-only types; nothing here
// crosses the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ssm {

// Forms of the decay's gate and of the input's weight (template parameters of the kernels).
enum { kGateRaw = 0, kGateSoftplus = 1, kGateSigmoid = 2 };
enum { kInputPlain = 0, kInputNorm = 1, kInputComplement = 2 };

struct GatedLinearArgs {
  const void* x;          // [B, L, D], steps x_step elements apart
  const void* gate;       // [B, L, D]
  const void* igate;      // [B, L, D] or null
  const float* A;         // [D]
  const float* gbias;     // [D] or null
  const float* ibias;     // [D] or null
  const float* h0;        // [B, D] or null
  const int32_t* seqlens; // [B] or null
  void* y;                // [B, L, D]
  float* h_final;         // [B, D] or null
  float* states;          // what the backward needs, or null
  void* workspace;
  int64_t batch, seqlen, dim;
  int64_t x_step, gate_step, igate_step;
  int in_bf16, out_bf16, act, scale;
};

struct GatedLinearBwdArgs {
  GatedLinearArgs f;      // the forward's inputs (y and h_final unused; states given, or the workspace's)
  const float* dy;
  const float* dh_final;  // or null
  float* dx;
  float* dgate;
  float* digate;          // null without an input gate
  float* dA;
  float* dgbias;          // or null
  float* dibias;          // or null
  float* dh0;             // or null
};

// Weak: the validation front end also links without these kernels (a host-only
// build); a call that passes validation there reports a launch failure.
__attribute__((weak)) int launch_gated_linear(const GatedLinearArgs& a, void* stream);
__attribute__((weak)) int launch_gated_linear_update(const GatedLinearArgs& a, void* stream);  // h_final: the state
__attribute__((weak)) int launch_gated_linear_bwd(const GatedLinearBwdArgs& a, void* stream);

// Tiles of 64 channels and 64 steps, at most.
inline bool gated_linear_fits(int64_t batch, int64_t seqlen, int64_t dim) {
  return batch * ((dim + 63) / 64) * ((seqlen + 63) / 64) <= (int64_t(1) << 30);
}

inline size_t gated_linear_states_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  return static_cast<size_t>(batch * seqlen * dim) * 4;
}
inline size_t gated_linear_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

// Parts of dA, dgate_bias and dinput_bias, one a batch row, and the states when they are not given.
inline size_t gated_linear_parts_bytes(int64_t batch, int64_t dim) {
  return (static_cast<size_t>(batch * dim) * 3 * 8 + 255) & ~size_t(255);
}
inline size_t gated_linear_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool have_states) {
  return gated_linear_parts_bytes(batch, dim) + (have_states ? 0 : gated_linear_states_bytes(batch, seqlen, dim));
}

}  // namespace ssm
