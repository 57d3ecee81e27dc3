// Root-mean-square norm of rows with the residual's addition, and its
// gradients.
//
//   s = x + residual;  y = s r w,  r = 1 / sqrt(mean(s^2) + eps)
//   8-bit output: scale = max|y| / 448 (a row), y / scale in e4m3
//   ds = r (u - s r mean(u s r)) + dresidual,  u = dy w;  dw = sum_rows dy s r
//
// Bounded by HBM: a row crosses it once. A row lives in the registers of its
// threads between the sum and the output (and, for the 8-bit output, between
// the row's largest value and the output): one wave per row up to 1024
// elements, four rows a block; above, a block of four waves per row with one
// LDS exchange per sum. A thread holds 8 elements a piece, NPK pieces; pieces
// are 16 bytes of bfloat16 or 32 of float32, consecutive threads read
// consecutive pieces. Measured: (32768, 4096) bfloat16 with a float32 residual 294
// us, 5.5 TB/s; (8192, 2560) to 8 bits 30 us, 4.9 TB/s; gradients of (32768, 4096)
// 372 us, 5.8 TB/s; a large copy reaches 5.1. (Rows that are not whole 16-byte pieces: one element a
// load, consecutive threads consecutive elements.)
#include <hip/hip_runtime.h>

#include "device_math.h"
#include "rms_norm.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;

// Eight elements of a row that starts at `at`: e, e + step .. e + 7 step (VEC:
// step 1); zeros past `dim`.
template <bool BF16, bool VEC, int STEP>
__device__ __forceinline__ void load8(const void* base, int64_t at, int e, int dim, float (&o)[8]) {
  if constexpr (VEC) {
    if (e < dim) {  // dim is a multiple of 8
      if constexpr (BF16) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at + e);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[2 * i] = __uint_as_float(u[i] << 16);
          o[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
      } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + e);
        const float4 a = q[0], b = q[1];
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
        o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = e + i * STEP < dim ? load_elem<BF16>(base, at + e + i * STEP) : 0.0f;
  }
}

template <bool BF16, bool VEC, int STEP>
__device__ __forceinline__ void store8(void* base, int64_t at, int e, int dim, const float (&v)[8]) {
  if constexpr (VEC) {
    if (e < dim) {
      if constexpr (BF16) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i])) |
                 (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i + 1])) << 16);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at + e) = make_uint4(u[0], u[1], u[2], u[3]);
      } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(base) + at + e);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (e + i * STEP < dim) store_elem<BF16>(base, at + e + i * STEP, v[i]);
    }
  }
}

// Eight values in e4m3 (already divided by the row's scale; what rounding took
// past 448 is brought back, NaN stays).
template <bool VEC, int STEP>
__device__ __forceinline__ void store8_e4m3(void* base, int64_t at, int e, int dim, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] > 448.0f ? 448.0f : (v[i] < -448.0f ? -448.0f : v[i]);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  uint8_t* dst = static_cast<uint8_t*>(base) + at + e;
  if constexpr (VEC) {
    if (e < dim) *reinterpret_cast<int2*>(dst) = make_int2(lo, hi);
  } else {
    const uint64_t w = static_cast<uint32_t>(lo) | (static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (e + i * STEP < dim) dst[i * STEP] = static_cast<uint8_t>(w >> (8 * i));
    }
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
// (a NaN is not seen by the largest value; it reaches the output itself)
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// Over the threads of a row: one wave (TPR = 64) or the block. `slot` is an
// LDS area of its own for each call in a kernel's pass over a row.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (slot[0] + slot[1]) + (slot[2] + slot[3]);
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ float row_max(float v, float* slot) {
  v = wave_max(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = fmaxf(fmaxf(slot[0], slot[1]), fmaxf(slot[2], slot[3]));
  }
  return v;
}

// OUT: 0 float32, 1 bfloat16, 2 e4m3. RES: 0 none, 1 float32, 2 bfloat16.
template <int TPR, int NPK, bool BF16_IN, int RES, int OUT, bool VEC>
__global__ __launch_bounds__(kThreads) void rms_norm_kernel(const RmsNormArgs p) {
  constexpr int STEP = VEC ? 1 : TPR;
  __shared__ float slots[2][4];
  const int dim = static_cast<int>(p.dim);
  const int t = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  if (row >= p.rows) return;  // whole waves; a block of one row is never cut
  const int64_t at = row * dim;
  float s[NPK][8];
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NPK; ++i) {
    const int e = VEC ? (i * TPR + t) * 8 : i * TPR * 8 + t;
    load8<BF16_IN, VEC, STEP>(p.x, at, e, dim, s[i]);
    if constexpr (RES != 0) {
      float r[8];
      load8<RES == 2, VEC, STEP>(p.residual, at, e, dim, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s[i][k] += r[k];
        // the norm is taken of what the stream holds
        if constexpr (RES == 2) s[i][k] = bf16_bits_to_f32(f32_to_bf16_bits(s[i][k]));
      }
      store8<RES == 2, VEC, STEP>(p.residual_out, at, e, dim, s[i]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sq = fmaf(s[i][k], s[i][k], sq);
  }
  float r = rsqrtf(row_sum<TPR>(sq, slots[0]) / static_cast<float>(dim) + p.eps);
  // 8 bits: the rows are first taken with the power of two in r alone, so that
  // y = n / scale is one rounding of s w and one of a factor, and what r was
  // rounded by stands in the scale only. (With n, the scale's inverse and their
  // product, two roundings more, more elements came out as the other neighbour.)
  float rest = 1.0f;
  if constexpr (OUT == 2) {
    const uint32_t bits = __float_as_uint(r);
    const bool normal = (bits >> 23) > 0 && (bits >> 23) < 255;
    if (normal) {
      rest = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
      r = __uint_as_float(bits & 0x7f800000u);
    }
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < NPK; ++i) {
    const int e = VEC ? (i * TPR + t) * 8 : i * TPR * 8 + t;
    float w[8];
    if (p.weight != nullptr) {
      load8<false, VEC, STEP>(p.weight, 0, e, dim, w);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 1.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s[i][k] = s[i][k] * r * w[k];
      if constexpr (OUT == 2) top = fmaxf(top, fabsf(s[i][k]));
    }
    if constexpr (OUT != 2) store8<OUT == 1, VEC, STEP>(p.y, at, e, dim, s[i]);
  }
  if constexpr (OUT == 2) {
    top = row_max<TPR>(top, slots[1]);
    float scale = top * rest / 448.0f, inv = 448.0f / top;
    if (!(scale >= 0x1p-126f)) {  // (under 2^-128 a scale has no finite inverse; 1 for a row of zeros)
      scale = top > 0.0f ? 0x1p-126f : 1.0f;
      inv = rest / scale;
    }
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) s[i][k] *= inv;
      store8_e4m3<VEC, STEP>(p.y, at, VEC ? (i * TPR + t) * 8 : i * TPR * 8 + t, dim, s[i]);
    }
    if (t == 0) p.scales[row] = scale;
  }
}

// Gradients. A block takes every gridDim.x-th row (or four rows, one a wave)
// and keeps its part of dweight in registers; the parts are added by
// rms_norm_dweight_kernel in block order.
template <int TPR, int NPK, bool BF16, bool VEC>
__global__ __launch_bounds__(kThreads) void rms_norm_bwd_kernel(const RmsNormBwdArgs p) {
  constexpr int kRows = kThreads / TPR, STEP = VEC ? 1 : TPR;
  __shared__ float slots[4][4];
  const int dim = static_cast<int>(p.dim);
  const int t = threadIdx.x % TPR, part = threadIdx.x / TPR;
  float dw[NPK][8], w[NPK][8];
#pragma unroll
  for (int i = 0; i < NPK; ++i) {
    const int e = VEC ? (i * TPR + t) * 8 : i * TPR * 8 + t;
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = 0.0f, w[i][k] = 1.0f;
    if (p.weight != nullptr) load8<false, VEC, STEP>(p.weight, 0, e, dim, w[i]);
  }
  int pass = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + part; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows, pass ^= 1) {
    const int64_t at = row * dim;
    float s[NPK][8], g[NPK][8];
    float sq = 0.0f, su = 0.0f;
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
      const int e = VEC ? (i * TPR + t) * 8 : i * TPR * 8 + t;
      load8<BF16, VEC, STEP>(p.s, at, e, dim, s[i]);
      load8<false, VEC, STEP>(p.dy, at, e, dim, g[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sq = fmaf(s[i][k], s[i][k], sq);
        su = fmaf(g[i][k] * w[i][k], s[i][k], su);
      }
    }
    // two slots a pass, two passes in turn: a slot is written again only
    // behind the next pass's barriers
    sq = row_sum<TPR>(sq, slots[2 * pass]);
    su = row_sum<TPR>(su, slots[2 * pass + 1]);
    const float r = rsqrtf(sq / static_cast<float>(dim) + p.eps);
    const float c = su / static_cast<float>(dim) * r * r;
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
      const int e = VEC ? (i * TPR + t) * 8 : i * TPR * 8 + t;
      float o[8];
      if (p.dresidual != nullptr) {
        load8<false, VEC, STEP>(p.dresidual, at, e, dim, o);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dw[i][k] = fmaf(g[i][k], s[i][k] * r, dw[i][k]);
        o[k] = fmaf(r, fmaf(-s[i][k], c, g[i][k] * w[i][k]), o[k]);
      }
      store8<false, VEC, STEP>(p.ds, at, e, dim, o);
    }
  }
  if (p.dweight == nullptr) return;
  float* out = static_cast<float*>(p.workspace);
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
      store8<false, VEC, STEP>(out, static_cast<int64_t>(blockIdx.x) * dim, VEC ? (i * TPR + t) * 8 : i * TPR * 8 + t, dim, dw[i]);
    }
  } else {
    __shared__ float sums[kRows][NPK * 8 * TPR];
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) sums[part][(i * 8 + k) * TPR + t] = dw[i][k];
    }
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = (i * 8 + k) * TPR + t;
          dw[i][k] = (sums[0][at] + sums[1][at]) + (sums[2][at] + sums[3][at]);
        }
        store8<false, VEC, STEP>(out, static_cast<int64_t>(blockIdx.x) * dim, VEC ? (i * TPR + t) * 8 : i * TPR * 8 + t, dim, dw[i]);
      }
    }
  }
}

// dweight[c] = sum over the blocks' parts: 64 columns a block, sixteen waves
// each adding every sixteenth part, then the sixteen sums in order. (Four waves
// took 7.4 us for 500 parts of 1537: too few loads in flight.)
constexpr int kDwWaves = 16;
__global__ __launch_bounds__(64 * kDwWaves) void rms_norm_dweight_kernel(const float* __restrict__ parts, int nparts,
                                                                         int dim, float* __restrict__ dweight) {
  __shared__ float sums[kDwWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = static_cast<int>(blockIdx.x) * 64 + lane;
  float acc = 0.0f;
  if (c < dim) {
    int i = w;
    for (; i + 7 * kDwWaves < nparts; i += 8 * kDwWaves) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = parts[static_cast<int64_t>(i + k * kDwWaves) * dim + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc += v[k];
    }
    for (; i < nparts; i += kDwWaves) acc += parts[static_cast<int64_t>(i) * dim + c];
  }
  sums[w][lane] = acc;
  __syncthreads();
  if (w == 0 && c < dim) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kDwWaves; ++k) v += sums[k][lane];
    dweight[c] = v;
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// f(threads per row, pieces a thread) for a row of `dim` elements.
template <typename F>
void by_width(int64_t dim, F&& f) {
  using std::integral_constant;
  if (dim <= 512) {
    f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  } else if (dim <= 1024) {
    f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  } else if (dim <= 2048) {
    f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  } else if (dim <= 4096) {
    f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  } else if (dim <= 8192) {
    f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  } else {
    f(integral_constant<int, 256>{}, integral_constant<int, 8>{});
  }
}

template <bool BI, int RES, int OUT>
void launch_norm(const RmsNormArgs& a, bool vec, hipStream_t st) {
  by_width(a.dim, [&](auto tpr, auto npk) {
    constexpr int TPR = decltype(tpr)::value, NPK = decltype(npk)::value;
    const unsigned blocks = static_cast<unsigned>((a.rows + kThreads / TPR - 1) / (kThreads / TPR));
    if (vec) {
      rms_norm_kernel<TPR, NPK, BI, RES, OUT, true><<<blocks, kThreads, 0, st>>>(a);
    } else {
      rms_norm_kernel<TPR, NPK, BI, RES, OUT, false><<<blocks, kThreads, 0, st>>>(a);
    }
  });
}

template <bool BI, int RES>
void launch_norm_out(const RmsNormArgs& a, bool vec, hipStream_t st) {
  if (a.out_type == 0) {
    launch_norm<BI, RES, 0>(a, vec, st);
  } else if (a.out_type == 1) {
    launch_norm<BI, RES, 1>(a, vec, st);
  } else {
    launch_norm<BI, RES, 2>(a, vec, st);
  }
}

template <bool BI>
void launch_norm_res(const RmsNormArgs& a, bool vec, hipStream_t st) {
  if (a.residual == nullptr) {
    launch_norm_out<BI, 0>(a, vec, st);
  } else if (a.res_bf16) {
    launch_norm_out<BI, 2>(a, vec, st);
  } else {
    launch_norm_out<BI, 1>(a, vec, st);
  }
}

}  // namespace

int launch_rms_norm(const RmsNormArgs& all, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  // 2^23 rows a launch: up to as many blocks, which stay below 2^32 threads.
  constexpr int64_t kRowsALaunch = int64_t(1) << 23;
  const auto behind = [](const void* p, int64_t bytes) {
    return p != nullptr ? const_cast<char*>(static_cast<const char*>(p)) + bytes : nullptr;
  };
  for (int64_t row = 0; row < all.rows; row += kRowsALaunch) {
    RmsNormArgs a = all;
    const int64_t n = row * a.dim, res = n * (a.res_bf16 ? 2 : 4);
    a.rows = all.rows - row < kRowsALaunch ? all.rows - row : kRowsALaunch;
    a.x = behind(a.x, n * (a.in_bf16 ? 2 : 4));
    a.residual = behind(a.residual, res);
    a.residual_out = behind(a.residual_out, res);
    a.y = behind(a.y, n * (a.out_type == 0 ? 4 : (a.out_type == 1 ? 2 : 1)));
    a.scales = reinterpret_cast<float*>(behind(a.scales, row * 4));
    const bool vec = a.dim % 8 == 0 && on16(a.x) && on16(a.residual) && on16(a.weight) && on16(a.y) &&
                     on16(a.residual_out);
    a.in_bf16 ? launch_norm_res<true>(a, vec, st) : launch_norm_res<false>(a, vec, st);
    if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  }
  return 0;
}

int launch_rms_norm_bwd(const RmsNormBwdArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool vec = a.dim % 8 == 0 && on16(a.s) && on16(a.weight) && on16(a.dy) && on16(a.dresidual) && on16(a.ds);
  int nparts = 0;
  if (a.rows > 0) {
    nparts = static_cast<int>(rms_norm_bwd_blocks(a.rows, a.dim));
    by_width(a.dim, [&](auto tpr, auto npk) {
      constexpr int TPR = decltype(tpr)::value, NPK = decltype(npk)::value;
      const unsigned blocks = static_cast<unsigned>(nparts);
      if (a.s_bf16) {
        vec ? rms_norm_bwd_kernel<TPR, NPK, true, true><<<blocks, kThreads, 0, st>>>(a)
            : rms_norm_bwd_kernel<TPR, NPK, true, false><<<blocks, kThreads, 0, st>>>(a);
      } else {
        vec ? rms_norm_bwd_kernel<TPR, NPK, false, true><<<blocks, kThreads, 0, st>>>(a)
            : rms_norm_bwd_kernel<TPR, NPK, false, false><<<blocks, kThreads, 0, st>>>(a);
      }
    });
    if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  }
  if (a.dweight != nullptr) {
    const unsigned blocks = static_cast<unsigned>((a.dim + 63) / 64);
    rms_norm_dweight_kernel<<<blocks, 64 * kDwWaves, 0, st>>>(static_cast<const float*>(a.workspace), nparts,
                                                         static_cast<int>(a.dim), a.dweight);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
