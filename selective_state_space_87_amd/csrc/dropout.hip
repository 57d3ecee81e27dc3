// Dropout with the residual's addition, and its gradient (the same product with
// the same bits, which are drawn again, never stored).
//
//   y = residual + x keep / (1 - p)
//
// A thread takes eight consecutive elements, the half words of one block of the
// generator. Bounded by HBM, the bits being drawn while the loads are under way:
// (32768, 4096) bfloat16 with a float32 residual 230 us, 5.8 TB/s (a large copy
// reaches 5.1), (17052, 2560) bfloat16 without one 29 us, 6.0 TB/s; (1000, 1537)
// float32 4.3 us.
#include <hip/hip_runtime.h>

#include "layer_norm.h"
#include "philox.h"
#include "rows.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;

template <bool BF16_IN, bool RES, bool BF16_OUT>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const DropoutArgs p) {
  const DropKey key = drop_key(p.drop.rng, p.drop.call, p.drop.threshold, p.drop.scale);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads * 8;
  const auto piece = [&](int64_t e, int left) __attribute__((always_inline)) {
    float v[8], r[8];
    load_piece<BF16_IN>(p.x, e, left, v);
    if constexpr (RES) load_piece<BF16_OUT>(p.residual, e, left, r);
    drop8(key, static_cast<uint64_t>(e), v);
    if constexpr (RES) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += r[k];
    }
    store_piece<BF16_OUT>(p.y, e, left, v);
  };
  for (int64_t e = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 8; e < p.n; e += step) {
    if (p.n - e >= 8) {
      piece(e, 8);  // no branch on the way: the loads are under way while the bits are drawn
    } else {
      piece(e, static_cast<int>(p.n - e));
    }
  }
}

template <bool BI, bool RES>
void launch(const DropoutArgs& a, unsigned blocks, hipStream_t st) {
  a.out_bf16 ? dropout_kernel<BI, RES, true><<<blocks, kThreads, 0, st>>>(a)
             : dropout_kernel<BI, RES, false><<<blocks, kThreads, 0, st>>>(a);
}

}  // namespace

int launch_dropout(const DropoutArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t groups = (a.n + kThreads * 8 - 1) / (kThreads * 8);
  constexpr int64_t kMostBlocks = int64_t(1) << 20;  // (below 2^32 threads)
  const unsigned blocks = static_cast<unsigned>(groups < kMostBlocks ? groups : kMostBlocks);
  if (a.residual != nullptr) {
    a.in_bf16 ? launch<true, true>(a, blocks, st) : launch<false, true>(a, blocks, st);
  } else {
    a.in_bf16 ? launch<true, false>(a, blocks, st) : launch<false, false>(a, blocks, st);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
