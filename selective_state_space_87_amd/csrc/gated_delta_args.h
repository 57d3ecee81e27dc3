// Interface between the C-ABI front end (api.cpp) and the gated delta rule's
// launchers, and the plan of a call. Host-only types; nothing here crosses the
// public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ssm {

struct GatedDeltaArgs {
  const void* q;          // [B, L, G, N], steps q_step elements apart
  const void* k;          // [B, L, G, N]
  const void* v;          // [B, L, H, P]
  const void* dt;         // [B, L, H]
  const float* A;         // [H]
  const void* beta;       // [B, L, H]
  const float* dt_bias;   // [H] or null
  const float* h0;        // [B, H, P, N] or null
  const int32_t* seqlens; // [B] or null
  void* y;                // [B, L, H, P]
  float* h_final;         // [B, H, P, N] or null
  void* workspace;
  int64_t batch, seqlen, nkheads, nheads, headdim, dstate;
  int64_t q_step, k_step, v_step;
  float scale;
  int in_bf16, out_bf16, dt_softplus, beta_sigmoid, qk_l2norm;
};

struct GatedDeltaBwdArgs {
  GatedDeltaArgs f;       // the forward's inputs (y and h_final unused)
  const float* dy;
  const float* dh_final;
  float* dq;
  float* dk;
  float* dv;
  float* ddt;
  float* dA;
  float* dbeta;
  float* ddt_bias;
  float* dh0;
};

constexpr int64_t kGdrMaxHeadDim = 256;
constexpr int64_t kGdrMaxState = 128;
constexpr float kGdrMinLogDecay = -200.0f;  // exp of it is 0 in float32
constexpr float kL2NormEps = 1e-6f;

// Weak: the validation front end also links without these kernels (a host-only
// build with stand-ins for the scan's launchers); a call that passes
// validation there reports a launch failure.
__attribute__((weak)) int launch_gated_delta(const GatedDeltaArgs& a, void* stream);
__attribute__((weak)) int launch_gated_delta_update(const GatedDeltaArgs& a, void* stream);  // h_final: the state
__attribute__((weak)) int launch_gated_delta_bwd(const GatedDeltaBwdArgs& a, void* stream);

// How a gated delta rule of given sizes runs forward: as a plain recurrence
// (one launch, no workspace) or in chunks of 64 steps, with the workspace
// holding the chunks' triangular inverses, output weights, keys and queries
// (halves) and per-step factors. A pure function of the sizes.
struct GdrPlan {
  bool recurrent;
  int64_t chunks;  // per batch row
  // Forward of few heads and many chunks: `segs` segments of seg_chunks chunks,
  // walked at the same time from states that a pass before has found.
  int64_t segs, seg_chunks;
  size_t off_map, off_seg;
  size_t off_t, off_p, off_k, off_q, off_fac;
  size_t off_tt, off_s, off_x, off_e, off_top, off_part;  // backward only
  size_t bytes;
};
// Up to this length the recurrence is taken: its time grows with the steps, a
// chunk's does not. Measured (bf16, N = P = 128, chunks against recurrence) at 4, 8
// and 16 steps: 2 heads 19 us against 19, 20, 33; 256 heads 39 against 25, 34, 42;
// 2048 heads 208 to 218 against 95, 169, 319.
constexpr int64_t kGdrRecurrentSteps = 8;
// Segments: with at most kGdrFewSlices slices of 16 columns (batch, heads and
// head size together) the walks of whole sequences leave most of the device
// idle, and finding the segments' states first (a pass over P + N columns in
// place of P) costs less than it gives. As many segments as make
// kGdrManySlices slices, 4 to 32, of at least kGdrSegChunks chunks. Measured
// (bf16, N = P = 128, whole -> in segments): 1 head of 65536 steps 1785 -> 218
// us, 8 heads 2136 -> 684, 16 heads (128 slices) 2337 -> 1308, 32 heads 2639 -> 2785
// (not taken); 16 heads of 16384 steps 594 -> 365, 4 of 4096 133 -> 79, 2 of 2048
// 76 -> 58 (in two segments 80).
constexpr int64_t kGdrFewSlices = 128, kGdrManySlices = 1024, kGdrSegChunks = 8, kGdrMinSegs = 4, kGdrMaxSegs = 32;
inline GdrPlan plan_gated_delta(int64_t batch, int64_t seqlen, int64_t nkheads, int64_t nheads, int64_t headdim,
                                int64_t dstate, int in_bf16, bool backward) {
  GdrPlan p{};
  p.recurrent = !backward && (seqlen <= kGdrRecurrentSteps || batch == 0 || nheads == 0);
  if (p.recurrent) return p;
  p.chunks = (seqlen + 63) / 64;
  if (p.chunks == 0 || batch == 0 || nheads == 0) {  // (backward of nothing)
    p.segs = p.seg_chunks = 1;
    return p;
  }
  const size_t items = static_cast<size_t>(batch * nheads * p.chunks);
  constexpr size_t kPieces = 6 * 2 * 64 * 8 * 2;  // bytes of T's (or the weights') halves a chunk
  size_t at = 0;
  const auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const auto take_n = [&](size_t n, size_t bytes) {
    const size_t here = at;
    at = (at + n * bytes + 255) & ~size_t(255);
    return here;
  };
  const auto take = [&](size_t item_bytes) { return take_n(items, item_bytes); };
  p.off_t = take(kPieces);
  p.off_p = take(kPieces);
  const size_t kv_items = static_cast<size_t>(batch * nkheads * p.chunks);
  const size_t kv = (in_bf16 ? 1 : 2) * 64 * (dstate <= 64 ? 64 : 128) * 2;
  p.off_k = take_n(kv_items, kv);
  p.off_q = take_n(kv_items, kv);
  p.off_fac = take(9 * 64 * 4);
  p.segs = 1;
  const int64_t slices = batch * nheads * ceil_div(headdim, 16);
  if (!backward && slices <= kGdrFewSlices) {
    int64_t n = kGdrManySlices / slices;
    if (n > kGdrMaxSegs) n = kGdrMaxSegs;
    if (n > p.chunks / kGdrSegChunks) n = p.chunks / kGdrSegChunks;
    if (n >= kGdrMinSegs) p.segs = n;
  }
  p.seg_chunks = ceil_div(p.chunks, p.segs);
  p.segs = ceil_div(p.chunks, p.seg_chunks);
  if (p.segs > 1) {
    const size_t heads = static_cast<size_t>(batch * nheads);
    p.off_map = take_n(heads * static_cast<size_t>(p.segs), static_cast<size_t>((headdim + dstate) * dstate) * 4);
    p.off_seg = take_n(heads * static_cast<size_t>(p.segs), static_cast<size_t>(headdim * dstate) * 4);
  }
  if (backward) {
    const size_t state = static_cast<size_t>(headdim * dstate) * 4;
    p.off_tt = take(kPieces);
    p.off_s = take(state);
    p.off_x = take(state);
    p.off_e = take(static_cast<size_t>(64 * headdim) * 4);
    p.off_top = take(5 * 32 * 4);
    p.off_part = take(2 * 8);
  }
  p.bytes = at;
  return p;
}

inline size_t gated_delta_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nkheads, int64_t nheads,
                                          int64_t headdim, int64_t dstate, int in_bf16) {
  return plan_gated_delta(batch, seqlen, nkheads, nheads, headdim, dstate, in_bf16, false).bytes;
}

inline size_t gated_delta_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nkheads, int64_t nheads,
                                              int64_t headdim, int64_t dstate, int in_bf16) {
  return plan_gated_delta(batch, seqlen, nkheads, nheads, headdim, dstate, in_bf16, true).bytes;
}

}  // namespace ssm
