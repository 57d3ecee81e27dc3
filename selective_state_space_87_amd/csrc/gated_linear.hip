// Gated linear recurrence: the step-by-step kernel (single tokens and short
// sequences), and the launchers; the tiles of long sequences are in
// gated_linear_{fwd,bwd}.h.
#include <hip/hip_runtime.h>

#include "column_sums.h"
#include "gated_linear_tile.h"

namespace ssm {

namespace {

// A thread walks four channels of a batch row, the next step's inputs on their way
// while one is taken.
template <bool BF16, int ACT, int SCALE, bool GATED>
__global__ __launch_bounds__(kGlrThreads) void glr_walk_kernel(const GatedLinearArgs p) {
  constexpr int VC = 4;
  const int64_t per_row = (p.dim + VC - 1) / VC;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kGlrThreads + threadIdx.x;
  if (i >= p.batch * per_row) return;
  const int64_t b = i / per_row;
  const int c = static_cast<int>(i - b * per_row) * VC, left = static_cast<int>(p.dim) - c;
  const int64_t steps = gdr_row_steps(p.seqlens, static_cast<int>(b), p.seqlen);
  GlrParams<VC, ACT, GATED> par;
  GlrRaw<BF16, GATED, VC, 1> raw;
  if (steps > 0) raw.load(p, b * p.seqlen, c, left, 0, 1, left >= VC);
  par.load(p, c, left);
  float h[VC] = {};
  if (p.h0 != nullptr) glr_load_f32<VC>(p.h0, b * p.dim + c, left, h);
  if (p.states != nullptr && p.seqlen > 0) glr_store<false, VC>(p.states, b * p.dim + c, left, h);
  for (int64_t t = 0; t < p.seqlen; ++t) {
    float y[VC] = {};
    if (t < steps) {
      const GlrRaw<BF16, GATED, VC, 1> now = raw;
      if (t + 1 < steps) raw.load(p, b * p.seqlen + t + 1, c, left, 0, 1, left >= VC);
      float a[1][VC], in[1][VC];
      glr_elements<BF16, ACT, SCALE, GATED, 1, VC>(now, par, a, in);
#pragma unroll
      for (int v = 0; v < VC; ++v) y[v] = h[v] = fmaf(a[0][v], h[v], in[0][v]);
    }
    if (p.y != nullptr) {
      const int64_t to = (b * p.seqlen + t) * p.dim + c;
      if (p.out_bf16) {
        glr_store<true, VC>(p.y, to, left, y);
      } else {
        glr_store<false, VC>(p.y, to, left, y);
      }
    }
  }
  if (p.h_final != nullptr) glr_store<false, VC>(p.h_final, b * p.dim + c, left, h);
}

template <bool BF16>
void launch_walk(const GatedLinearArgs& a, hipStream_t st) {
  const int64_t threads = a.batch * ((a.dim + 3) / 4);
  const unsigned blocks = static_cast<unsigned>((threads + kGlrThreads - 1) / kGlrThreads);
  glr_by_form(a, [&](auto act, auto scale, auto gated) {
    glr_walk_kernel<BF16, decltype(act)::value, decltype(scale)::value, decltype(gated)::value>
        <<<blocks, kGlrThreads, 0, st>>>(a);
  });
}

__global__ __launch_bounds__(kGlrThreads) void glr_clear_kernel(uint4* words, int64_t counts, int64_t n) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGlrThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kGlrThreads + threadIdx.x; i < n; i += step) {
    const uint32_t v = i < counts ? 0u : kGlrMissing;
    words[i] = make_uint4(v, v, v, v);
  }
}

}  // namespace

void launch_glr_clear(const GlrChainPlan& p, void* workspace, hipStream_t st) {
  const int64_t n = static_cast<int64_t>(p.bytes / 16);
  const int64_t blocks = (n + kGlrThreads - 1) / kGlrThreads;
  glr_clear_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), kGlrThreads, 0, st>>>(
      static_cast<uint4*>(workspace), static_cast<int64_t>(p.off_words / 16), n);
}

int launch_gated_linear(const GatedLinearArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (gated_linear_walks(a.batch, a.seqlen, a.dim)) {
    a.in_bf16 ? launch_walk<true>(a, st) : launch_walk<false>(a, st);
  } else {
    const GlrChainPlan plan = plan_glr_chain(a.batch, a.seqlen, a.dim, kGlrFwdSteps);
    a.in_bf16 ? launch_glr_fwd<true>(a, plan, st) : launch_glr_fwd<false>(a, plan, st);
  }
  return static_cast<int>(hipGetLastError());
}

int launch_gated_linear_update(const GatedLinearArgs& given, void* stream) {
  GatedLinearArgs a = given;
  a.h0 = a.h_final;
  return launch_gated_linear(a, stream);
}

int launch_gated_linear_bwd(const GatedLinearBwdArgs& given, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  GatedLinearBwdArgs a = given;
  const GlrBwdPlan plan = plan_gated_linear_bwd(a.f.batch, a.f.seqlen, a.f.dim, a.f.states != nullptr);
  if (a.f.batch > 0) {
    if (a.f.states == nullptr) {
      a.f.states = reinterpret_cast<float*>(static_cast<char*>(a.f.workspace) + plan.off_states);
      if (const int e = launch_gated_linear(a.f, stream)) return e;
    }
    a.f.in_bf16 ? launch_glr_bwd<true>(a, plan, st) : launch_glr_bwd<false>(a, plan, st);
    if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  }
  launch_column_sums(static_cast<const char*>(a.f.workspace) + plan.off_parts, a.f.batch * plan.chain.tiles, 3 * a.f.dim,
                     StoreRows<3>{{a.dA, a.dgbias, a.dibias}, a.f.dim}, st);
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
