// Rows of float32 or bfloat16 in pieces of eight consecutive elements, for the
// layer norm and the dropout. A whole piece is one 16-byte access (two for
// float32) at whatever boundary the row starts on: rows of odd widths start
// anywhere, and the memory unit takes any boundary. A piece that the row ends
// in goes element by element.
#pragma once

#include <hip/hip_runtime.h>

#include "device_math.h"

namespace ssm {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// Elements at .. at + 7 of `base`, of which the row holds `left` (zeros past those).
template <bool BF16>
__device__ __forceinline__ void load_piece(const void* base, int64_t at, int left, float (&o)[8]) {
  if (left >= 8) {
    if constexpr (BF16) {
      const u32x4_any u = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(u[i] << 16);
        o[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
      const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(base) + at);
      const f32x4_any a = q[0], b = q[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = a[i], o[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = i < left ? load_elem<BF16>(base, at + i) : 0.0f;
  }
}

template <bool BF16>
__device__ __forceinline__ void store_piece(void* base, int64_t at, int left, const float (&v)[8]) {
  if (left >= 8) {
    if constexpr (BF16) {
      u32x4_any u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i])) |
               (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i + 1])) << 16);
      }
      *reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(base) + at) = u;
    } else {
      f32x4_any* q = reinterpret_cast<f32x4_any*>(static_cast<float*>(base) + at);
      q[0] = f32x4_any{v[0], v[1], v[2], v[3]};
      q[1] = f32x4_any{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < left) store_elem<BF16>(base, at + i, v[i]);
    }
  }
}

// Sums of N values over the threads of a row: a wave (TPR = 64) or the block.
// A kernel gives each of its sums a `slots` area of its own; with two sums or
// more a row, an area is written again only behind another sum's barrier.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*slots)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v[i] += __shfl_xor(v[i], m);
  }
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slots[threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = slots[0][i];
#pragma unroll
      for (int w = 1; w < TPR / 64; ++w) t += slots[w][i];
      v[i] = t;
    }
  }
}

}  // namespace ssm
