// Gradients of the causal depthwise conv1d + SiLU (conv1d.hip), for gfx950.
//
// Per batch row b, channel d, step l, filter width K, with the inputs before
// step 0 from the carried state (or zero):
//   out[l] = bias + sum_k w[k] x[l - (K-1) + k];  y = silu(out)
//   g[l]   = dy[l] silu'(out[l])                   (out is computed again)
//   dx[l]  = sum_k w[k] g[l + K-1 - k]             (l < 0: the carried state's)
//   dw[k]  = sum_{b,l} g[l] x[l - (K-1) + k];  dbias = sum_{b,l} g[l]
//
// Bounded by HBM: x and dy are read once, dx written once. As forward, a thread
// has VC = 4 adjacent channels and walks a segment of steps with the last K
// inputs and the last K values of g in registers (circular: after unrolling by
// K nothing moves). dx[l] is complete K - 1 steps after l, so a segment walks
// K - 1 steps past its end; those steps' g is the next segment's too, but only
// the step's own segment counts it in dw. Measured: (4, 8192, 4096, width 4)
// bfloat16 245 us and 4.6 us for the sums, 5.4 TB/s of x, dy and dx (a large copy
// reaches 5.1); (2, 777, 333, width 3) float32 11 and 3.9 us, some five loads' chains.
// The width is a compile-time one: taps
// of zero in front of a narrower filter would make 0 * infinity of what they meet.
#include <hip/hip_runtime.h>

#include "column_sums.h"
#include "conv1d_bwd.h"
#include "device_math.h"

namespace ssm {

namespace {

// Any element boundary: rows of odd widths start anywhere, and the memory unit
// takes all. x and dy stream through once, dx too: past the caches.
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kBlock = 64;

template <int VC, bool BF16>
__device__ __forceinline__ void load_in(const void* base, int64_t i, float (&v)[VC]) {
  if constexpr (VC == 4 && BF16) {
    const u32x2_any r =
        __builtin_nontemporal_load(reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(base) + i));
    v[0] = __uint_as_float(r.x << 16);
    v[1] = __uint_as_float(r.x & 0xffff0000u);
    v[2] = __uint_as_float(r.y << 16);
    v[3] = __uint_as_float(r.y & 0xffff0000u);
  } else if constexpr (VC == 4) {
    const f32x4_any r =
        __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(static_cast<const float*>(base) + i));
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = r[c];
  } else {
    v[0] = load_elem<BF16>(base, i);
  }
}

template <int VC>
__device__ __forceinline__ void store_out(float* p, const float (&v)[VC]) {
  if constexpr (VC == 4) {
    __builtin_nontemporal_store(f32x4_any{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4_any*>(p));
  } else {
    p[0] = v[0];
  }
}

// silu'(z) = s (1 + z (1 - s)), s = 1 / (1 + e^-z); 1 - s = e^-z s. (e^-z is
// infinite below z = -88: s and the derivative are 0 there, as s z is.)
__device__ __forceinline__ float silu_slope(float z) {
  const float e = exp2_hw(-z * kLog2e), s = rcp_hw(1.0f + e);
  return z < -80.0f ? 0.0f : s * fmaf(z, e * s, 1.0f);
}

template <int K, int VC, bool BF16, bool SILU>
__global__ __launch_bounds__(kBlock) void conv1d_bwd_kernel(const ConvBwdArgs a, int seg) {
  constexpr int kGroup = K * (K < 8 ? 8 / K : 1);  // steps whose loads are issued together
  const int64_t L = a.seqlen, Dm = a.dim;
  int64_t c0 = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) * VC;
  if (c0 >= Dm) return;
  // The last thread of an odd width takes the last VC channels, some of them its
  // neighbour's too: both find, and write, the same values.
  if (c0 > Dm - VC) c0 = Dm - VC;
  const int64_t b = blockIdx.z;
  const int64_t row0 = b * L;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * seg;
  const int64_t t1 = t0 + seg < L ? t0 + seg : L;

  float w[K][VC], bv[VC], dw[K][VC], db[VC];
  float dw2[K][VC] = {}, db2[VC] = {};  // the segment's sums, to which dw and db go every group of steps
#pragma unroll
  for (int c = 0; c < VC; ++c) {
    bv[c] = a.bias ? a.bias[c0 + c] : 0.0f;
    db[c] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][c] = a.weight[(c0 + c) * K + k], dw[k][c] = 0.0f;
  }

  // Slot s of the windows holds the step that is s modulo K past t0.
  float x[K][VC], g[K][VC];
#pragma unroll
  for (int j = 1; j < K; ++j) {
    const int64_t t = t0 - K + j;
    if (t >= 0) {
      load_in<VC, BF16>(a.x, (row0 + t) * Dm + c0, x[j]);
    } else {  // t0 = 0: the carried state's slot K - 1 + t
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        x[j][c] = a.state_in && K - 1 + t >= 0 ? a.state_in[(b * Dm + c0 + c) * (K - 1) + (K - 1 + t)] : 0.0f;
      }
    }
#pragma unroll
    for (int c = 0; c < VC; ++c) g[j][c] = 0.0f;
  }
  // One step: x[u] holds its input, d its dy; l = t - (K - 1) is complete.
  const auto step = [&](int64_t t, int u, const float (&d)[VC], bool live, bool own, bool emit)
                        __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < VC; ++c) {
      float out = bv[c];
#pragma unroll
      for (int k = 0; k < K; ++k) out = fmaf(w[k][c], x[(u + 1 + k) % K][c], out);
      g[u][c] = live ? (SILU ? d[c] * silu_slope(out) : d[c]) : 0.0f;
    }
    if (own) {
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        db[c] += g[u][c];
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][c] = fmaf(g[u][c], x[(u + 1 + k) % K][c], dw[k][c]);
      }
    }
    if (emit) {
      const int64_t l = t - (K - 1);
      float o[VC];
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        o[c] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) o[c] = fmaf(w[k][c], g[(u + K - k) % K][c], o[c]);  // g[t - k]
      }
      const int64_t j = l - (L - (K - 1));  // the carried-out state's slot of input l
      if (j >= 0 && a.dstate_out) {
#pragma unroll
        for (int c = 0; c < VC; ++c) o[c] += a.dstate_out[(b * Dm + c0 + c) * (K - 1) + j];
      }
      if (l >= 0) {
        store_out<VC>(a.dx + (row0 + l) * Dm + c0, o);
      } else if (a.dstate_in) {
#pragma unroll
        for (int c = 0; c < VC; ++c) a.dstate_in[(b * Dm + c0 + c) * (K - 1) + (K - 1) + l] = o[c];
      }
    }
  };
  // N steps from t on, of which the last may lie past the end, where there is no
  // output: g is 0. All loads come before the first step, those past the end from
  // the last row: no branch stands between them.
  const auto edges = [&](int64_t t, auto head) __attribute__((always_inline)) {
    constexpr bool kHead = decltype(head)::value;  // the segment's first steps, else those behind the groups
    float in[K][VC], d[K][VC];
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const int64_t row = row0 + (t + u < L ? t + u : L - 1);
      load_in<VC, BF16>(a.x, row * Dm + c0, in[u]);
      load_in<VC, false>(a.dy, row * Dm + c0, d[u]);
    }
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const bool live = t + u < L;
#pragma unroll
      for (int c = 0; c < VC; ++c) x[u][c] = live ? in[u][c] : 0.0f;
      // the first K - 1 steps complete nothing of the segment's own: at the sequence's
      // start the carried state's inputs
      if (kHead || t + u < t1 + K - 1) step(t + u, u, d[u], live, t + u < t1, !kHead || u == K - 1 || t0 == 0);
    }
  };

  // A sum takes a rounding for every group and one for every step of a group, not one for
  // every step of a segment.
  const auto fold = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < VC; ++c) {
      db2[c] += db[c], db[c] = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) dw2[k][c] += dw[k][c], dw[k][c] = 0.0f;
    }
  };

  if (L > 0) {  // (then t0 < t1)
    edges(t0, std::true_type{});
    fold();
    int64_t t = t0 + K;
    for (; t + kGroup <= t1; t += kGroup) {
      float in[kGroup][VC], d[kGroup][VC];
#pragma unroll
      for (int u = 0; u < kGroup; ++u) load_in<VC, BF16>(a.x, (row0 + t + u) * Dm + c0, in[u]);
#pragma unroll
      for (int u = 0; u < kGroup; ++u) load_in<VC, false>(a.dy, (row0 + t + u) * Dm + c0, d[u]);
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
#pragma unroll
        for (int c = 0; c < VC; ++c) x[u % K][c] = in[u][c];
        step(t + u, u % K, d[u], true, true, true);
      }
      fold();
    }
    // What is left of the segment, and the K - 1 steps behind it that complete its last dx.
    for (; t < t1 + K - 1; t += K) edges(t, std::false_type{});
    fold();
  } else if (a.dstate_in) {  // no step: the state has passed through
#pragma unroll
    for (int c = 0; c < VC; ++c) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int64_t at = (b * Dm + c0 + c) * (K - 1) + j;
        a.dstate_in[at] = a.dstate_out ? a.dstate_out[at] : 0.0f;
      }
    }
  }

  if (a.dweight == nullptr && a.dbias == nullptr) return;
  // parts [batch row, segment][k, then bias][channel]
  float* part = static_cast<float*>(a.workspace) + (b * gridDim.y + blockIdx.y) * (K + 1) * Dm + c0;
#pragma unroll
  for (int c = 0; c < VC; ++c) {
#pragma unroll
    for (int k = 0; k < K; ++k) part[k * Dm + c] = dw2[k][c];
    part[K * Dm + c] = db2[c];
  }
}

// Columns [k, then bias][channel] of the parts: dweight is [channel][k].
struct StoreFilters {
  float* dweight;
  float* dbias;
  int64_t dim, width;

  __device__ __forceinline__ void operator()(int64_t c, float v) const {
    const int64_t k = c / dim, d = c - k * dim;
    if (k < width) {
      if (dweight != nullptr) dweight[d * width + k] = v;
    } else if (dbias != nullptr) {
      dbias[d] = v;
    }
  }
};

template <int K, bool BF16>
void launch_width(const ConvBwdArgs& a, const ConvBwdPlan& p, hipStream_t st) {
  const int vc = a.dim >= 4 ? 4 : 1;
  const int64_t groups = (a.dim + vc - 1) / vc;
  const dim3 grid(static_cast<unsigned>((groups + kBlock - 1) / kBlock), static_cast<unsigned>(p.segs),
                  static_cast<unsigned>(a.batch));
  const int seg = static_cast<int>(p.seg);
  if (vc == 4) {
    a.silu ? conv1d_bwd_kernel<K, 4, BF16, true><<<grid, kBlock, 0, st>>>(a, seg)
           : conv1d_bwd_kernel<K, 4, BF16, false><<<grid, kBlock, 0, st>>>(a, seg);
  } else {
    a.silu ? conv1d_bwd_kernel<K, 1, BF16, true><<<grid, kBlock, 0, st>>>(a, seg)
           : conv1d_bwd_kernel<K, 1, BF16, false><<<grid, kBlock, 0, st>>>(a, seg);
  }
}

template <bool BF16>
void launch_type(const ConvBwdArgs& a, const ConvBwdPlan& p, hipStream_t st) {
  switch (a.width) {
    case 1: return launch_width<1, BF16>(a, p, st);
    case 2: return launch_width<2, BF16>(a, p, st);
    case 3: return launch_width<3, BF16>(a, p, st);
    case 4: return launch_width<4, BF16>(a, p, st);
    case 5: return launch_width<5, BF16>(a, p, st);
    case 6: return launch_width<6, BF16>(a, p, st);
    case 7: return launch_width<7, BF16>(a, p, st);
    default: return launch_width<8, BF16>(a, p, st);
  }
}

}  // namespace

int launch_conv1d_bwd(const ConvBwdArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const ConvBwdPlan p = plan_conv1d_bwd(a.batch, a.seqlen, a.dim, a.width);
  if (a.batch > 0) {
    a.in_bf16 ? launch_type<true>(a, p, st) : launch_type<false>(a, p, st);
    if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  }
  if (a.dweight != nullptr || a.dbias != nullptr) {
    launch_column_sums(a.workspace, a.batch * p.segs, (a.width + 1) * a.dim,
                       StoreFilters{a.dweight, a.dbias, a.dim, a.width}, st);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
