// Backward tiles of the gated linear recurrence; instantiated for bfloat16 and
// float32 inputs in gated_linear_bwd_{b,f}.hip. See gated_linear_tile.h.
//
// With E the gradient that reaches a step's state from behind, D = E + dy, and a D
// reaches the state before: the maps E -> P E + R of slices and tiles join from
// the last to the first, over the same products P of decays as forward. A tile
// (64 steps) has the state that enters it from the forward, takes both
// recurrences through its slices at once, and computes its gates a second time
// where the gradients are formed: the inputs stay in registers, what was made of
// them would not fit. Its sums over steps are one part a tile, joined in double
// in a fixed order (column_sums.h).
//
// Bounded by HBM: (8, 2048, 1536) bfloat16 with both gates 115 us, 4.8 TB/s of the
// inputs, dy and the three gradients, 115 instructions an element; four channels a thread (eight, whose float32
// gradients go in two stores each: 179 us with an earlier chain, four 134).
#pragma once

#include "gated_linear_tile.h"

namespace ssm {

template <bool BF16, int ACT, int SCALE, bool GATED, bool CHAIN>
__global__ __launch_bounds__(kGlrThreads) void glr_bwd_kernel(const GatedLinearBwdArgs q, const GlrChain chain,
                                                              const uint32_t tiles, float* parts) {
  constexpr int VC = 4;
  using Shape = GlrShape<VC, kGlrBwdSteps>;
  constexpr int SL = Shape::kSlices, TS = Shape::kSteps, kRun = Shape::kRun;
  __shared__ __attribute__((aligned(16))) float lp[SL][kGlrChannels], ls[SL][kGlrChannels], lr[SL][kGlrChannels];
  __shared__ float rp[kGlrRuns][kGlrChannels], rs[kGlrRuns][kGlrChannels], rr[kGlrRuns][kGlrChannels];
  __shared__ float enter_h[kGlrChannels], enter_e[kGlrChannels];
  __shared__ uint32_t slot;
  const GatedLinearArgs& p = q.f;
  uint32_t k = 0, group = blockIdx.x;
  if constexpr (CHAIN) {
    k = glr_ticket<true>(chain, &slot, &group);
    if (k == kGlrNoTile) return;
  }
  const GlrGroup at = glr_group(p, group);
  const int64_t t0 = static_cast<int64_t>(k) * kGlrBwdSteps;
  const int slice = threadIdx.x / Shape::kLanes;
  const int ch = static_cast<int>(threadIdx.x % Shape::kLanes) * VC, c = at.c0 + ch;
  const int left = static_cast<int>(p.dim) - c;
  const int there = glr_steps_in(p.seqlen, t0, kGlrBwdSteps);
  const int n = glr_steps_in(at.steps, t0, there);
  const int lane = threadIdx.x % kGlrChannels, run = threadIdx.x / kGlrChannels, ce = at.c0 + lane;
  float* part = parts + (static_cast<int64_t>(at.b) * tiles + k) * 3 * p.dim;
  if (n <= 0) {  // behind the row's end: gradients of 0, and nobody waits for it
    const float zero[VC] = {};
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      const int64_t to = (at.row0 + t0 + slice * TS + i) * p.dim + c;
      if (slice * TS + i < there) {
        glr_store<false, VC>(q.dx, to, left, zero);
        glr_store<false, VC>(q.dgate, to, left, zero);
        if constexpr (GATED) glr_store<false, VC>(q.digate, to, left, zero);
      }
    }
    if (run == 0 && ce < p.dim) {
      if (there > 0) part[ce] = part[p.dim + ce] = part[2 * p.dim + ce] = 0.0f;
      const int64_t i = static_cast<int64_t>(at.b) * p.dim + ce;
      if (k == 0 && q.dh0 != nullptr) q.dh0[i] = q.dh_final != nullptr ? q.dh_final[i] : 0.0f;
    }
    return;
  }

  GlrRaw<BF16, GATED, VC, TS> raw;
  GlrParams<VC, ACT, GATED> par;
  float dy[TS][VC], a[TS][VC], b[TS][VC];
  const bool whole = n == kGlrBwdSteps && at.c0 + kGlrChannels <= p.dim;
  par.load(p, c, left);  // first, since loads come in order: what needs it need not wait for all of the tile
  // Each path computes for itself: where they have met all loads are waited for (training
  // step (8, 2048, 1536) 173.5 us for 170).
  const auto take = [&](auto all) __attribute__((always_inline)) {
    constexpr bool kAll = decltype(all)::value;
    raw.load(p, at.row0 + t0, c, left, slice * TS, n, kAll);
    const int64_t from = (at.row0 + t0 + slice * TS) * p.dim + c;
    typename GlrPack<false, VC>::Words d[TS];
#pragma unroll
    for (int i = 0; i < TS; ++i) d[i] = glr_load<false, VC>(q.dy, from + i * p.dim, kAll ? VC : (slice * TS + i < n ? left : 0));
    glr_elements<BF16, ACT, SCALE, GATED, TS, VC>(raw, par, a, b);
    if constexpr (!kAll) glr_mask<TS, VC>(slice * TS, n, a, b);
#pragma unroll
    for (int i = 0; i < TS; ++i) {
#pragma unroll
      for (int v = 0; v < VC; ++v) dy[i][v] = __uint_as_float(d[i][v]);
    }
  };
  if (whole) {
    take(std::true_type{});
  } else {
    take(std::false_type{});
  }
  {
    float P[VC], S[VC], R[VC];
#pragma unroll
    for (int v = 0; v < VC; ++v) {
      P[v] = 1.0f, S[v] = R[v] = 0.0f;
#pragma unroll
      for (int i = 0; i < TS; ++i) P[v] *= a[i][v], S[v] = fmaf(a[i][v], S[v], b[i][v]);
    }
#pragma unroll
    for (int i = TS - 1; i >= 0; --i) {
#pragma unroll
      for (int v = 0; v < VC; ++v) R[v] = a[i][v] * (dy[i][v] + R[v]);
    }
#pragma unroll
    for (int v = 0; v < VC; ++v) lp[slice][ch + v] = P[v], ls[slice][ch + v] = S[v], lr[slice][ch + v] = R[v];
  }
  __syncthreads();
  float sp[kRun], ss[kRun], sr[kRun];
  float rP = 1.0f, rS = 0.0f, rR = 0.0f;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    sp[i] = lp[run * kRun + i][lane], ss[i] = ls[run * kRun + i][lane], sr[i] = lr[run * kRun + i][lane];
    rP *= sp[i];
    rS = fmaf(sp[i], rS, ss[i]);
  }
#pragma unroll
  for (int i = kRun - 1; i >= 0; --i) rR = fmaf(sp[i], rR, sr[i]);
  rp[run][lane] = rP, rs[run][lane] = rS, rr[run][lane] = rR;
  __syncthreads();
  if (run == 0) {
    const int64_t i = static_cast<int64_t>(at.b) * p.dim + ce;
    float e = q.dh_final != nullptr && ce < p.dim ? q.dh_final[i] : 0.0f;
    enter_h[lane] = ce < p.dim ? p.states[(static_cast<int64_t>(at.b) * tiles + k) * p.dim + ce] : 0.0f;
    float P = 1.0f, R = 0.0f;
#pragma unroll
    for (int r = kGlrRuns - 1; r >= 0; --r) {
      P *= rp[r][lane];
      R = fmaf(rp[r][lane], R, rr[r][lane]);
    }
    if constexpr (CHAIN) {
      const uint32_t last = static_cast<uint32_t>((at.steps - 1) / kGlrBwdSteps);
      e = glr_enter(chain, group, last - k, P, R, e);
    }
    enter_e[lane] = e;
    if (k == 0 && q.dh0 != nullptr && ce < p.dim) q.dh0[i] = fmaf(P, e, R);
  }
  __syncthreads();
  {
    float h = enter_h[lane], e = enter_e[lane];
#pragma unroll
    for (int r = 0; r < kGlrRuns - 1; ++r) {
      if (r < run) h = fmaf(rp[r][lane], h, rs[r][lane]);
    }
#pragma unroll
    for (int r = kGlrRuns - 1; r > 0; --r) {
      if (r > run) e = fmaf(rp[r][lane], e, rr[r][lane]);
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      ls[run * kRun + i][lane] = h;
      h = fmaf(sp[i], h, ss[i]);
    }
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i) {
      lr[run * kRun + i][lane] = e;
      e = fmaf(sp[i], e, sr[i]);
    }
  }
  __syncthreads();

  raw.template forget<ACT>();
  float before[TS][VC], E[VC], sumA[VC], sumg[VC], sumi[VC];
#pragma unroll
  for (int v = 0; v < VC; ++v) {
    float h = ls[slice][ch + v];
    E[v] = lr[slice][ch + v];
    sumA[v] = sumg[v] = sumi[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      before[i][v] = h;
      h = fmaf(a[i][v], h, b[i][v]);
    }
  }
#pragma unroll
  for (int i = TS - 1; i >= 0; --i) {
    const int s = slice * TS + i;
    const bool on = s < n;
    float dx[VC], dg[VC], di[VC];
#pragma unroll
    for (int v = 0; v < VC; ++v) {
      const float D = dy[i][v] + E[v];
      float slope, islope = 0.0f, in = glr_elem<BF16>(raw.x[i], v), sig = 1.0f;
      const float g = gate_value_slope<ACT>(glr_elem<BF16>(raw.gate[i], v) + par.gbias[v], &slope);
      const float w = input_weight<SCALE>(par.A2[v] * g, a[i][v]);
      const float dv = on ? w * D : 0.0f;
      if constexpr (GATED) sig = glr_sigmoid_slope(glr_elem<BF16>(raw.igate[i], v) + par.ibias[v], &islope);
      dx[v] = dv * sig;
      di[v] = dv * in * islope;
      const float dla = on ? D * fmaf(a[i][v], before[i][v], input_weight_slope<SCALE>(a[i][v], w) * (in * sig)) : 0.0f;
      dg[v] = dla * (par.A2[v] * kLn2) * slope;
      sumA[v] = fmaf(dla, g, sumA[v]);
      sumg[v] += dg[v];
      sumi[v] += di[v];
      E[v] = a[i][v] * D;
    }
    if (s < there) {
      const int64_t to = (at.row0 + t0 + s) * p.dim + c;
      glr_store<false, VC>(q.dx, to, left, dx);
      glr_store<false, VC>(q.dgate, to, left, dg);
      if constexpr (GATED) glr_store<false, VC>(q.digate, to, left, di);
    }
  }
  __syncthreads();  // ls and lr have been read
#pragma unroll
  for (int v = 0; v < VC; ++v) lp[slice][ch + v] = sumA[v], ls[slice][ch + v] = sumg[v], lr[slice][ch + v] = sumi[v];
  __syncthreads();
  float total[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    total[0] += lp[run * kRun + i][lane];
    total[1] += ls[run * kRun + i][lane];
    total[2] += lr[run * kRun + i][lane];
  }
  rp[run][lane] = total[0], rs[run][lane] = total[1], rr[run][lane] = total[2];
  __syncthreads();
  if (run == 0 && ce < p.dim) {
    float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < kGlrRuns; ++r) sum[0] += rp[r][lane], sum[1] += rs[r][lane], sum[2] += rr[r][lane];
#pragma unroll
    for (int i = 0; i < 3; ++i) part[i * p.dim + ce] = sum[i];
  }
}

template <bool BF16>
void launch_glr_bwd(const GatedLinearBwdArgs& a, const GlrBwdPlan& plan, hipStream_t st) {
  const GlrChainPlan& cp = plan.chain;
  float* parts = reinterpret_cast<float*>(static_cast<char*>(a.f.workspace) + plan.off_parts);
  const uint32_t tiles = static_cast<uint32_t>(cp.tiles);
  glr_by_form(a.f, [&](auto act, auto scale, auto gated) {
    constexpr int ACT = decltype(act)::value, SCALE = decltype(scale)::value;
    constexpr bool GATED = decltype(gated)::value;
    if (cp.tiles > 1) {
      launch_glr_clear(cp, a.f.workspace, st);
      glr_bwd_kernel<BF16, ACT, SCALE, GATED, true><<<static_cast<unsigned>(cp.columns * cp.tiles), kGlrThreads, 0, st>>>(
          a, glr_chain(cp, a.f.workspace), tiles, parts);
    } else {
      glr_bwd_kernel<BF16, ACT, SCALE, GATED, false>
          <<<static_cast<unsigned>(cp.groups), kGlrThreads, 0, st>>>(a, GlrChain{}, tiles, parts);
    }
  });
}

}  // namespace ssm
