// Sums of a gradient's parts, one kernel for all operators that leave them: parts
// [nparts][cols], float32, written by blocks that each took some of the rows or steps.
//
// 64 columns a block, sixteen waves each adding every sixteenth part in double, eight
// loads at a time, then the sixteen sums in order: the same way in every run. It is a
// chain of loads that bounds it (98 to 512 parts 4 us).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace ssm {

constexpr int kSumWaves = 16;

// store(c, sum) puts the sum of column c, rounded once, where it belongs.
template <typename Store>
__global__ __launch_bounds__(64 * kSumWaves) void column_sums_kernel(const float* __restrict__ parts, int64_t nparts,
                                                                     int64_t cols, const Store store) {
  __shared__ double sums[kSumWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  double acc = 0.0;
  if (c < cols) {
    int64_t i = w;
    for (; i + 7 * kSumWaves < nparts; i += 8 * kSumWaves) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = parts[(i + k * kSumWaves) * cols + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc += v[k];
    }
    for (; i < nparts; i += kSumWaves) acc += parts[i * cols + c];
  }
  sums[w][lane] = acc;
  __syncthreads();
  if (w == 0 && c < cols) {
    double v = 0.0;
#pragma unroll
    for (int k = 0; k < kSumWaves; ++k) v += sums[k][lane];
    store(c, static_cast<float>(v));
  }
}

template <typename Store>
void launch_column_sums(const void* parts, int64_t nparts, int64_t cols, const Store& store, hipStream_t st) {
  column_sums_kernel<<<static_cast<unsigned>((cols + 63) / 64), 64 * kSumWaves, 0, st>>>(
      static_cast<const float*>(parts), nparts, cols, store);
}

// Columns of consecutive rows of `dim`, a row an output; NULL outputs are left out.
template <int N>
struct StoreRows {
  float* out[N];
  int64_t dim;

  __device__ __forceinline__ void operator()(int64_t c, float v) const {
    const int64_t row = c / dim;
    float* to = out[0];
#pragma unroll
    for (int i = 1; i < N; ++i) to = row == i ? out[i] : to;
    if (to != nullptr) to[c - row * dim] = v;
  }
};

}  // namespace ssm
