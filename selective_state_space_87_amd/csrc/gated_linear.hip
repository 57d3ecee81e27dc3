// Gated linear recurrence, forward, single token and backward: the plain form,
// one thread a batch row and channel, step by step.
#include <hip/hip_runtime.h>

#include "gated_linear.h"

namespace ssm {

namespace {

constexpr int kThreads = 64;

template <bool BF16, int ACT, int SCALE>
struct Element {
  float u, g, slope, la, a, w, x, s, s_slope, v;
  __device__ __forceinline__ Element(const GatedLinearArgs& p, int64_t row, int64_t d) {
    u = load_elem<BF16>(p.gate, row * p.gate_step + d) + (p.gbias ? p.gbias[d] : 0.0f);
    g = gate_value_slope<ACT>(u, &slope);
    la = p.A[d] * g;
    a = decay(la);
    w = input_weight<SCALE>(la, a);
    x = load_elem<BF16>(p.x, row * p.x_step + d);
    s = 1.0f, s_slope = 0.0f;
    if (p.igate) {
      s = sigmoid_slope(load_elem<BF16>(p.igate, row * p.igate_step + d) + (p.ibias ? p.ibias[d] : 0.0f), &s_slope);
    }
    v = x * s;
  }
};

__device__ __forceinline__ int64_t row_steps(const GatedLinearArgs& p, int64_t b) {
  return gdr_row_steps(p.seqlens, static_cast<int>(b), p.seqlen);
}

template <bool BF16, int ACT, int SCALE>
__global__ __launch_bounds__(kThreads) void gated_linear_kernel(const GatedLinearArgs p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.batch * p.dim) return;
  const int64_t b = i / p.dim, d = i - b * p.dim, steps = row_steps(p, b);
  float h = p.h0 ? p.h0[i] : 0.0f;
  for (int64_t t = 0; t < p.seqlen; ++t) {
    const int64_t at = (b * p.seqlen + t) * p.dim + d;
    if (p.states) p.states[at] = h;
    if (t < steps) {
      const Element<BF16, ACT, SCALE> e(p, b * p.seqlen + t, d);
      h = fmaf(e.a, h, e.w * e.v);
    }
    if (p.y) {
      const float y = t < steps ? h : 0.0f;
      p.out_bf16 ? store_elem<true>(p.y, at, y) : store_elem<false>(p.y, at, y);
    }
  }
  if (p.h_final) p.h_final[i] = h;
}

template <bool BF16, int ACT, int SCALE>
__global__ __launch_bounds__(kThreads) void gated_linear_bwd_kernel(const GatedLinearBwdArgs q) {
  const GatedLinearArgs& p = q.f;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, n = p.batch * p.dim;
  if (i >= n) return;
  const int64_t b = i / p.dim, d = i - b * p.dim, steps = row_steps(p, b);
  float dh = q.dh_final ? q.dh_final[i] : 0.0f;
  double dA = 0.0, dgb = 0.0, dib = 0.0;
  for (int64_t t = p.seqlen - 1; t >= 0; --t) {
    const int64_t at = (b * p.seqlen + t) * p.dim + d;
    float dx = 0.0f, dg = 0.0f, di = 0.0f;
    if (t < steps) {
      const Element<BF16, ACT, SCALE> e(p, b * p.seqlen + t, d);
      dh += q.dy[at];
      const float dv = e.w * dh;
      dx = dv * e.s;
      di = dv * e.x * e.s_slope;
      const float dla = dh * fmaf(e.a, p.states[at], input_weight_slope<SCALE>(e.a, e.w) * e.v);
      dg = dla * p.A[d] * e.slope;
      dA += dla * e.g;
      dgb += dg;
      dib += di;
      dh *= e.a;
    }
    q.dx[at] = dx;
    q.dgate[at] = dg;
    if (q.digate) q.digate[at] = di;
  }
  if (q.dh0) q.dh0[i] = dh;
  double* parts = static_cast<double*>(p.workspace);
  parts[i] = dA, parts[n + i] = dgb, parts[2 * n + i] = dib;
}

__global__ __launch_bounds__(kThreads) void gated_linear_sums_kernel(const GatedLinearBwdArgs q) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, n = q.f.batch * q.f.dim;
  if (d >= q.f.dim) return;
  const double* parts = static_cast<const double*>(q.f.workspace);
  float* out[3] = {q.dA, q.dgbias, q.dibias};
  for (int k = 0; k < 3; ++k) {
    double sum = 0.0;
    for (int64_t i = d; i < n; i += q.f.dim) sum += parts[k * n + i];
    if (out[k]) out[k][d] = static_cast<float>(sum);
  }
}

// One token: the step above, in place on the state.
template <bool BF16, int ACT, int SCALE>
__global__ __launch_bounds__(kThreads) void gated_linear_update_kernel(const GatedLinearArgs p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.batch * p.dim) return;
  const int64_t b = i / p.dim, d = i - b * p.dim;
  const Element<BF16, ACT, SCALE> e(p, b, d);
  const float h = fmaf(e.a, p.h_final[i], e.w * e.v);
  p.h_final[i] = h;
  p.out_bf16 ? store_elem<true>(p.y, i, h) : store_elem<false>(p.y, i, h);
}

// f(in_bf16, act, scale) as compile-time constants.
template <typename F>
void by_form(const GatedLinearArgs& p, F&& f) {
  using std::integral_constant;
  const auto scale = [&](auto bf16, auto act) {
    if (p.scale == kInputNorm) {
      f(bf16, act, integral_constant<int, kInputNorm>{});
    } else if (p.scale == kInputComplement) {
      f(bf16, act, integral_constant<int, kInputComplement>{});
    } else {
      f(bf16, act, integral_constant<int, kInputPlain>{});
    }
  };
  const auto act = [&](auto bf16) {
    if (p.act == kGateSigmoid) {
      scale(bf16, integral_constant<int, kGateSigmoid>{});
    } else if (p.act == kGateSoftplus) {
      scale(bf16, integral_constant<int, kGateSoftplus>{});
    } else {
      scale(bf16, integral_constant<int, kGateRaw>{});
    }
  };
  p.in_bf16 ? act(std::true_type{}) : act(std::false_type{});
}

unsigned blocks_of(int64_t n) { return static_cast<unsigned>((n + kThreads - 1) / kThreads); }

}  // namespace

int launch_gated_linear(const GatedLinearArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  by_form(a, [&](auto bf16, auto act, auto scale) {
    gated_linear_kernel<decltype(bf16)::value, decltype(act)::value, decltype(scale)::value>
        <<<blocks_of(a.batch * a.dim), kThreads, 0, st>>>(a);
  });
  return static_cast<int>(hipGetLastError());
}

int launch_gated_linear_update(const GatedLinearArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  by_form(a, [&](auto bf16, auto act, auto scale) {
    gated_linear_update_kernel<decltype(bf16)::value, decltype(act)::value, decltype(scale)::value>
        <<<blocks_of(a.batch * a.dim), kThreads, 0, st>>>(a);
  });
  return static_cast<int>(hipGetLastError());
}

int launch_gated_linear_bwd(const GatedLinearBwdArgs& given, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  GatedLinearBwdArgs a = given;
  if (a.f.batch > 0) {
    if (a.f.states == nullptr) {
      GatedLinearArgs f = a.f;
      f.y = nullptr;
      f.h_final = nullptr;
      f.states = reinterpret_cast<float*>(static_cast<char*>(a.f.workspace) +
                                          gated_linear_parts_bytes(a.f.batch, a.f.dim));
      if (const int e = launch_gated_linear(f, stream)) return e;
      a.f.states = f.states;
    }
    by_form(a.f, [&](auto bf16, auto act, auto scale) {
      gated_linear_bwd_kernel<decltype(bf16)::value, decltype(act)::value, decltype(scale)::value>
          <<<blocks_of(a.f.batch * a.f.dim), kThreads, 0, st>>>(a);
    });
    if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  }
  gated_linear_sums_kernel<<<blocks_of(a.f.dim), kThreads, 0, st>>>(a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
