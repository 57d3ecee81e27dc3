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

// A long sequence runs in tiles of 64 channels, kGlrFwdSteps steps forward and
// kGlrBwdSteps backward, a block each. A tile's part of the recurrence is a pair
// (product of the decays, state from a zero start) a channel; a chain in the
// workspace joins the pairs (gated_linear_tile.h): a word a tile and channel, and
// one for every kGlrWindow tiles. Measured at (4, 8192, 4096) and (1, 65536, 2560)
// bfloat16: tiles of 64 steps 229 and 363 us, of 128 steps 214 and 295 (backward 64
// steps are what 142 to 157 registers hold); windows of 2, 3, 4, 5, 8, 16 tiles 215, 215, 214,
// 216, 217, 230 us and 310, 300, 295, 294, 292, 312.
constexpr int kGlrChannels = 64, kGlrFwdSteps = 128, kGlrBwdSteps = 64, kGlrWindow = 4;
constexpr int kGlrTicketBytes = 64;  // a count of its own line for every group

// The tile that a ticket is for: the first tiles first, backward the last first.
// kGlrNoTile for a ticket past the last tile, whatever it is: two calls at once that
// have been given the same workspace draw from one count, or find another call's words there.
constexpr uint32_t kGlrNoTile = 0xffffffffu;
constexpr uint32_t glr_tile_of(uint32_t ticket, uint32_t tiles, bool back) {
  return ticket >= tiles ? kGlrNoTile : (back ? tiles - 1 - ticket : ticket);
}

// How many of `steps` steps lie in the tile of `size` steps from t0 on: at most size, 0
// or less where they end before it. (A tile that glr_tile_of gives starts below 2^30, as
// sequences are shorter: the difference fits 32 bits.)
constexpr int glr_steps_in(int64_t steps, int64_t t0, int size) {
  return steps - t0 < size ? static_cast<int>(steps - t0) : size;
}

// Whether a sequence is walked step by step instead, a thread four channels: a step
// takes 0.5 us however few the channels are, a tile as long for 1 step as for 64,
// but blocks of many tiles are mostly idle. Measured, walked against tiles (us in the
// kernel, bfloat16): 1 x 2560 channels, 8, 12, 16, 64 steps 5.8, 7.6, 9.6, 32 against 9
// throughout; 16 x 2560 6.5, 8.4, 10, 39 against 15; 128 x 4096 10, 14, 17, 65 against 100
// (float32, 64 steps: 93 against 110).
inline bool gated_linear_walks(int64_t batch, int64_t seqlen, int64_t dim) {
  const int64_t groups = batch * ((dim + kGlrChannels - 1) / kGlrChannels);
  return seqlen <= 12 || (seqlen <= kGlrBwdSteps && seqlen <= groups / 64);
}

// At most as many blocks of 256 threads as keep a launch below 2^32 threads (the
// groups of channels are rounded up to a multiple of 8, see GlrChainPlan).
inline bool gated_linear_fits(int64_t batch, int64_t seqlen, int64_t dim) {
  const int64_t tiles = (seqlen + kGlrBwdSteps - 1) / kGlrBwdSteps;
  const int64_t groups = (batch * ((dim + kGlrChannels - 1) / kGlrChannels) + 7) / 8 * 8;
  return groups * (tiles > 0 ? tiles : 1) < (int64_t(1) << 24);
}

struct GlrChainPlan {
  int64_t groups, tiles;  // blocks of channels, over the batch rows; tiles of steps
  int64_t columns;        // groups, rounded up to one for each of the 8 XCDs
  size_t off_words, off_states, bytes;
};

inline GlrChainPlan plan_glr_chain(int64_t batch, int64_t seqlen, int64_t dim, int steps) {
  GlrChainPlan p{};
  p.groups = batch * ((dim + kGlrChannels - 1) / kGlrChannels);
  p.tiles = (seqlen + steps - 1) / steps;
  p.columns = (p.groups + 7) / 8 * 8;
  if (p.tiles <= 1) return p;
  const size_t word = static_cast<size_t>(p.groups) * kGlrChannels * 8;
  p.off_words = static_cast<size_t>(p.groups) * kGlrTicketBytes;
  p.off_states = p.off_words + static_cast<size_t>(p.tiles) * word;
  p.bytes = p.off_states + static_cast<size_t>(p.tiles / kGlrWindow) * word;
  return p;
}

// States entering every tile of kGlrBwdSteps steps, [B, tiles, D] float32.
inline size_t gated_linear_states_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  return static_cast<size_t>(batch * ((seqlen + kGlrBwdSteps - 1) / kGlrBwdSteps) * dim) * 4;
}

inline size_t gated_linear_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  return plan_glr_chain(batch, seqlen, dim, kGlrFwdSteps).bytes;
}

// Backward: the chain (the forward's too, when the states are not given), the
// states, and a tile's parts of dA, dgate_bias and dinput_bias.
struct GlrBwdPlan {
  GlrChainPlan chain;
  size_t off_parts, off_states, bytes;
};

inline GlrBwdPlan plan_gated_linear_bwd(int64_t batch, int64_t seqlen, int64_t dim, bool have_states) {
  GlrBwdPlan p{};
  const auto align = [](size_t n) { return (n + 255) & ~size_t(255); };
  p.chain = plan_glr_chain(batch, seqlen, dim, kGlrBwdSteps);
  size_t chain = p.chain.bytes;
  if (!have_states) {
    const size_t fwd = gated_linear_workspace_bytes(batch, seqlen, dim);
    if (fwd > chain) chain = fwd;
  }
  p.off_parts = align(chain);
  p.off_states = p.off_parts + align(static_cast<size_t>(p.chain.tiles * batch * dim) * 3 * 4);
  p.bytes = p.off_states + (have_states ? 0 : align(gated_linear_states_bytes(batch, seqlen, dim)));
  return p;
}

inline size_t gated_linear_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool have_states) {
  return plan_gated_linear_bwd(batch, seqlen, dim, have_states).bytes;
}

}  // namespace ssm
