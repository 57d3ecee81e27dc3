// Forward tiles of the gated linear recurrence; instantiated for bfloat16 and
// float32 inputs in gated_linear_fwd_{b,f}.hip. See gated_linear_tile.h.
//
// Bounded by HBM: (4, 8192, 4096) bfloat16 with both gates 210 us, 5.1 TB/s, as a large
// copy; (1, 65536, 2560) 286 us, where 40 groups of channels are chains of 512 tiles,
// 4.7 TB/s. Vector work is 45 instructions an element, 0.74 of the time. The decays
// and inputs of a thread's 32 elements stay in registers while the tile waits
// for the state that enters it; what hides that wait, and the loads, are the other
// blocks of the CU: four of 128 registers (with earlier gates, at 239 us: three of 136 252,
// five, spilling, 252; blocks that stay and load the next tile while one waits, three of
// 168 registers, 295).
#pragma once

#include "gated_linear_tile.h"

namespace ssm {

template <bool BF16, int ACT, int SCALE, bool GATED, bool CHAIN>
__global__ __launch_bounds__(kGlrThreads, 4) void glr_fwd_kernel(const GatedLinearArgs p, const GlrChain chain) {
  constexpr int VC = BF16 ? 8 : 4;
  using Shape = GlrShape<VC, kGlrFwdSteps>;
  constexpr int SL = Shape::kSlices, TS = Shape::kSteps, kRun = Shape::kRun;
  __shared__ __attribute__((aligned(16))) float lp[SL][kGlrChannels], ls[SL][kGlrChannels];
  __shared__ float rp[kGlrRuns][kGlrChannels], rs[kGlrRuns][kGlrChannels], enter[kGlrChannels];
  __shared__ uint32_t slot;
  uint32_t k = 0, group = blockIdx.x;
  if constexpr (CHAIN) {
    k = glr_ticket<false>(chain, &slot, &group);
    if (k == kGlrNoTile) return;
  }
  const GlrGroup at = glr_group(p, group);
  const int64_t t0 = static_cast<int64_t>(k) * kGlrFwdSteps;
  const int slice = threadIdx.x / Shape::kLanes;
  const int c = at.c0 + static_cast<int>(threadIdx.x % Shape::kLanes) * VC;
  const int left = static_cast<int>(p.dim) - c;
  const int there = glr_steps_in(p.seqlen, t0, kGlrFwdSteps);  // steps of the array
  const int n = glr_steps_in(at.steps, t0, there);             // of the batch row
  int cy = c;
  const auto put = [&](int s, int wide, const float (&v)[VC]) __attribute__((always_inline)) {
    const int64_t to = (at.row0 + t0 + s) * p.dim + cy;
    if (p.out_bf16) {
      glr_store<true, VC>(p.y, to, wide, v);
    } else {
      glr_store<false, VC>(p.y, to, wide, v);
    }
  };
  if (n <= 0 && k > 0) {  // behind the row's end: nothing here, and nobody waits for it
    if (p.y != nullptr) {
      const float zero[VC] = {};
#pragma unroll
      for (int i = 0; i < TS; ++i) {
        if (slice * TS + i < there) put(slice * TS + i, left, zero);
      }
    }
    return;
  }

  float a[TS][VC], b[TS][VC], P[VC], S[VC];
  const bool whole = n == kGlrFwdSteps && at.c0 + kGlrChannels <= p.dim;
  {
    GlrRaw<BF16, GATED, VC, TS> raw;
    GlrParams<VC, ACT, GATED> par;
    par.load(p, c, left);  // first, since loads come in order: the first step's gates need not wait for the last's
    // In the chain a tile that is whole computes on its own path: where two paths have
    // met all loads are waited for ((4, 8192, 4096) bfloat16 212 us for 220). Of a sequence
    // in one tile that costs more registers than it gains (60 rows of 100 steps 62 us for 57).
    if (CHAIN && whole) {
      raw.load(p, at.row0 + t0, c, left, slice * TS, n, true);
      glr_elements<BF16, ACT, SCALE, GATED, TS, VC>(raw, par, a, b);
    } else {
      raw.load(p, at.row0 + t0, c, left, slice * TS, n, !CHAIN && whole);
      glr_elements<BF16, ACT, SCALE, GATED, TS, VC>(raw, par, a, b);
      if (CHAIN || !whole) glr_mask<TS, VC>(slice * TS, n, a, b);
    }
  }
#pragma unroll
  for (int v = 0; v < VC; ++v) {
    P[v] = 1.0f, S[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < TS; ++i) P[v] *= a[i][v], S[v] = fmaf(a[i][v], S[v], b[i][v]);
  }

  const int ch = c - at.c0;
#pragma unroll
  for (int v = 0; v < VC; ++v) lp[slice][ch + v] = P[v], ls[slice][ch + v] = S[v];
  __syncthreads();
  // 64 channels, four runs of slices
  const int lane = threadIdx.x % kGlrChannels, run = threadIdx.x / kGlrChannels;
  float sp[kRun], ss[kRun];
  float rP = 1.0f, rS = 0.0f;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    sp[i] = lp[run * kRun + i][lane], ss[i] = ls[run * kRun + i][lane];
    rP *= sp[i];
    rS = fmaf(sp[i], rS, ss[i]);
  }
  rp[run][lane] = rP, rs[run][lane] = rS;
  __syncthreads();
  if (run == 0) {
    const int ce = at.c0 + lane;
    float h = p.h0 != nullptr && ce < p.dim ? p.h0[static_cast<int64_t>(at.b) * p.dim + ce] : 0.0f;
    if constexpr (CHAIN) {
#pragma unroll
      for (int r = 1; r < kGlrRuns; ++r) {
        rP *= rp[r][lane];
        rS = fmaf(rp[r][lane], rS, rs[r][lane]);
      }
      h = glr_enter(chain, group, k, rP, rS, h);
    }
    enter[lane] = h;
  }
  __syncthreads();
  float h = enter[lane];
#pragma unroll
  for (int r = 0; r < kGlrRuns - 1; ++r) {
    if (r < run) h = fmaf(rp[r][lane], h, rs[r][lane]);
  }
  const int first = run * kRun * TS;  // step of the tile that the run starts with
  if (p.states != nullptr && first % kGlrBwdSteps == 0 && first < there && at.c0 + lane < p.dim) {
    const int64_t tiles = (p.seqlen + kGlrBwdSteps - 1) / kGlrBwdSteps;
    p.states[(at.b * tiles + (t0 + first) / kGlrBwdSteps) * p.dim + at.c0 + lane] = h;
  }
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    ls[run * kRun + i][lane] = h;
    h = fmaf(sp[i], h, ss[i]);
  }
  if (run == kGlrRuns - 1 && p.h_final != nullptr && t0 + n == at.steps && at.c0 + lane < p.dim) {
    p.h_final[static_cast<int64_t>(at.b) * p.dim + at.c0 + lane] = h;
  }
  __syncthreads();
  if (p.y == nullptr) return;
  asm volatile("" : "+v"(cy));  // y's addresses are made here, not kept from the loads on (some forms would spill)
#pragma unroll
  for (int v = 0; v < VC; ++v) S[v] = ls[slice][ch + v];
  if (whole) {
#pragma unroll
    for (int i = 0; i < TS; ++i) {
#pragma unroll
      for (int v = 0; v < VC; ++v) S[v] = fmaf(a[i][v], S[v], b[i][v]);
      put(slice * TS + i, VC, S);
    }
  } else {
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      const int s = slice * TS + i;
      float out[VC];
#pragma unroll
      for (int v = 0; v < VC; ++v) {
        S[v] = fmaf(a[i][v], S[v], b[i][v]);
        out[v] = s < n ? S[v] : 0.0f;
      }
      if (s < there) put(s, left, out);
    }
  }
}

template <bool BF16>
void launch_glr_fwd(const GatedLinearArgs& a, const GlrChainPlan& plan, hipStream_t st) {
  glr_by_form(a, [&](auto act, auto scale, auto gated) {
    constexpr int ACT = decltype(act)::value, SCALE = decltype(scale)::value;
    constexpr bool GATED = decltype(gated)::value;
    if (plan.tiles > 1) {
      launch_glr_clear(plan, a.workspace, st);
      glr_fwd_kernel<BF16, ACT, SCALE, GATED, true>
          <<<static_cast<unsigned>(plan.columns * plan.tiles), kGlrThreads, 0, st>>>(a, glr_chain(plan, a.workspace));
    } else {
      glr_fwd_kernel<BF16, ACT, SCALE, GATED, false>
          <<<static_cast<unsigned>(plan.groups), kGlrThreads, 0, st>>>(a, GlrChain{});
    }
  });
}

}  // namespace ssm
