// Layer norm of rows with the dropped-out residual addition, and its gradients.
//
//   s = drop(x) + residual;  d = s - mean(s);  y = d r weight + bias,
//   r = 1 / sqrt(mean(d^2) + eps)
//   u = dy weight, n = d r:  ds = r (u - mean(u) - n mean(u n)) + dresidual,
//   dx = drop(ds);  dweight = sum_rows dy n;  dbias = sum_rows dy
//
// Bounded by HBM: a row crosses it once and lives in the registers of its
// threads between the sums and the output: one wave a row up to 1024 elements,
// four rows a block; above, a block of 4, 8 or 16 waves a row. The mean is
// taken first, then the sums of the differences from it, their squares and
// (backward) their products: a row far from zero loses nothing, and what the
// first sum was rounded by is taken off as the mean of the differences. Blocks
// take rows in turn, the weights staying in their registers. Measured: (32768,
// 4096) bfloat16 with dropout and a float32 residual 295 us, 5.5 TB/s (a large copy
// reaches 5.1); gradients of (32768, 4096) with a float32 residual 385 to 405 us, 5.3
// to 5.6 TB/s; (1000, 1537) float32 10 us and 4 us for the sums. Streams past the caches
// (nontemporal) took 332 us forward, a next row on its way backward 415 us. Gradients of
// narrow rows are far from HBM's rate: at width 64, where 8 of a row's 64 lanes have data,
// 1.0 TB/s, at 128 1.9, from 512 on 5.4.
#include <hip/hip_runtime.h>

#include "column_sums.h"
#include "device_math.h"
#include "layer_norm.h"
#include "philox.h"
#include "rows.h"

namespace ssm {

namespace {

constexpr int block_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

// RES: 0 none, 1 float32, 2 bfloat16.
template <int TPR, int NPK, bool BF16_IN, int RES, bool BF16_OUT>
__global__ __launch_bounds__(block_threads(TPR)) void layer_norm_kernel(const LayerNormArgs p) {
  constexpr int kRows = block_threads(TPR) / TPR, kWaves = TPR / 64;
  __shared__ float sum_slots[kWaves][1], square_slots[kWaves][2];
  const int dim = static_cast<int>(p.dim);
  const int t = threadIdx.x % TPR;
  const float inv = 1.0f / static_cast<float>(dim);
  float w[NPK][8], bias[NPK][8];
#pragma unroll
  for (int i = 0; i < NPK; ++i) {
    const int e = (i * TPR + t) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) w[i][k] = 1.0f, bias[i][k] = 0.0f;
    if (p.weight != nullptr) load_piece<false>(p.weight, e, dim - e, w[i]);
    if (p.bias != nullptr) load_piece<false>(p.bias, e, dim - e, bias[i]);
  }
  DropKey key{};
  if (p.drop.threshold != 0) key = drop_key(p.drop.rng, p.drop.call, p.drop.threshold, p.drop.scale);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t at = row * dim;
    float s[NPK][8], sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
      const int e = (i * TPR + t) * 8;
      load_piece<BF16_IN>(p.x, at + e, dim - e, s[i]);
    }
    if constexpr (RES != 0) {
      float r[NPK][8];
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
        const int e = (i * TPR + t) * 8;
        load_piece<RES == 2>(p.residual, at + e, dim - e, r[i]);
      }
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
        const int e = (i * TPR + t) * 8;
        if (p.drop.threshold != 0 && e < dim) drop8(key, static_cast<uint64_t>(at + e), s[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s[i][k] += r[i][k];
          // the norm is taken of what the stream holds
          if constexpr (RES == 2) s[i][k] = bf16_bits_to_f32(f32_to_bf16_bits(s[i][k]));
        }
        store_piece<RES == 2>(p.residual_out, at + e, dim - e, s[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[0] += s[i][k];
    }
    row_sums<TPR>(sum, sum_slots);
    const float mean = sum[0] * inv;
    float sums[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
      const int left = dim - (i * TPR + t) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s[i][k] = k < left ? s[i][k] - mean : 0.0f;
        sums[0] += s[i][k];
        sums[1] = fmaf(s[i][k], s[i][k], sums[1]);
      }
    }
    row_sums<TPR>(sums, square_slots);
    const float rest = sums[0] * inv;
    const float var = fmaf(-rest, rest, sums[1] * inv);
    const float r = rsqrtf((var < 0.0f ? 0.0f : var) + p.eps);  // (NaN stays)
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
      const int e = (i * TPR + t) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) s[i][k] = fmaf((s[i][k] - rest) * r, w[i][k], bias[i][k]);
      store_piece<BF16_OUT>(p.y, at + e, dim - e, s[i]);
    }
  }
}

// Gradients. A block takes every gridDim.x-th row (or four rows, one a wave)
// and keeps its sums of dweight and dbias in registers. Every kLayerNormFold turns they
// are added to second sums, so that a sum takes that many roundings and one for every
// kLayerNormFold turns, not one a row. The second sums are registers too where four rows
// go to a block, where 64 turns may take no more than 100 us (10^6 rows of 64) and adding
// through the workspace 2; of longer rows, whose registers are full, they are the block's
// part in the workspace. The parts are added in block order (column_sums.h).
template <int TPR, int NPK, bool BF16>
__global__ __launch_bounds__(block_threads(TPR)) void layer_norm_bwd_kernel(const LayerNormBwdArgs p) {
  constexpr int kRows = block_threads(TPR) / TPR, kWaves = TPR / 64;
  __shared__ float sum_slots[kWaves][1], product_slots[kWaves][4];
  const int dim = static_cast<int>(p.dim);
  const int t = threadIdx.x % TPR, part = threadIdx.x / TPR;
  const float inv = 1.0f / static_cast<float>(dim);
  float dw[NPK][8], db[NPK][8], w[NPK][8];
#pragma unroll
  for (int i = 0; i < NPK; ++i) {
    const int e = (i * TPR + t) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = db[i][k] = 0.0f, w[i][k] = 1.0f;
    if (p.weight != nullptr) load_piece<false>(p.weight, e, dim - e, w[i]);
  }
  float dw2[NPK][8] = {}, db2[NPK][8] = {};  // (kRows > 1)
  DropKey key{};
  if (p.dx != nullptr && p.drop.threshold != 0) {
    key = drop_key(p.drop.rng, p.drop.call, p.drop.threshold, p.drop.scale);
  }
  // parts [block][dweight, dbias][dim]
  float* out = static_cast<float*>(p.workspace) + static_cast<int64_t>(blockIdx.x) * 2 * dim;
  // A piece of the part: written the first time, added to afterwards, by the same thread.
  const auto keep = [&](int at, int left, float (&v)[8], bool first) __attribute__((always_inline)) {
    if (!first) {
      float before[8];
      load_piece<false>(out, at, left, before);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += before[k];
    }
    store_piece<false>(out, at, left, v);
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  bool first = true;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + part; row < p.rows; first = false) {
    const int64_t fold = p.rows - row < kLayerNormFold * step ? p.rows : row + kLayerNormFold * step;
    for (; row < fold; row += step) {
      const int64_t at = row * dim;
      float s[NPK][8], g[NPK][8], o[NPK][8], sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
        const int e = (i * TPR + t) * 8;
        load_piece<BF16>(p.s, at + e, dim - e, s[i]);
      }
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
        const int e = (i * TPR + t) * 8;
        load_piece<false>(p.dy, at + e, dim - e, g[i]);
      }
      if (p.dresidual != nullptr) {
#pragma unroll
        for (int i = 0; i < NPK; ++i) {
          const int e = (i * TPR + t) * 8;
          load_piece<false>(p.dresidual, at + e, dim - e, o[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NPK; ++i) {
#pragma unroll
          for (int k = 0; k < 8; ++k) o[i][k] = 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[0] += s[i][k];
      }
      row_sums<TPR>(sum, sum_slots);
      const float mean = sum[0] * inv;
      float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // of d, d^2, u, u d
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
        const int left = dim - (i * TPR + t) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s[i][k] = k < left ? s[i][k] - mean : 0.0f;
          const float u = g[i][k] * w[i][k];
          sums[0] += s[i][k];
          sums[1] = fmaf(s[i][k], s[i][k], sums[1]);
          sums[2] += u;
          sums[3] = fmaf(u, s[i][k], sums[3]);
        }
      }
      row_sums<TPR>(sums, product_slots);
      const float rest = sums[0] * inv, mu = sums[2] * inv;
      const float var = fmaf(-rest, rest, sums[1] * inv);
      const float r = rsqrtf((var < 0.0f ? 0.0f : var) + p.eps);
      const float c = fmaf(-rest, mu, sums[3] * inv) * r;  // mean(u n)
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
        const int e = (i * TPR + t) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float n = (s[i][k] - rest) * r;
          dw[i][k] = fmaf(g[i][k], n, dw[i][k]);
          db[i][k] += g[i][k];
          o[i][k] = fmaf(r, fmaf(g[i][k], w[i][k], -mu) - n * c, o[i][k]);
        }
        store_piece<false>(p.ds, at + e, dim - e, o[i]);
        if (p.dx != nullptr && e < dim) {
          if (p.drop.threshold != 0) drop8(key, static_cast<uint64_t>(at + e), o[i]);
          store_piece<false>(p.dx, at + e, dim - e, o[i]);
        }
      }
    }
    if (p.dweight == nullptr && p.dbias == nullptr) continue;
#pragma unroll
    for (int i = 0; i < NPK; ++i) {
      if constexpr (kRows == 1) {
        const int e = (i * TPR + t) * 8;
        keep(e, dim - e, dw[i], first);
        keep(dim + e, dim - e, db[i], first);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (kRows > 1) dw2[i][k] += dw[i][k], db2[i][k] += db[i][k];
        dw[i][k] = db[i][k] = 0.0f;
      }
    }
  }
  if constexpr (kRows > 1) {
    if (p.dweight == nullptr && p.dbias == nullptr) return;
    __shared__ float adds[kRows][NPK * 8 * TPR];
    const auto add = [&](float (&v)[NPK][8], int to) {
#pragma unroll
      for (int i = 0; i < NPK; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) adds[part][(i * 8 + k) * TPR + t] = v[i][k];
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int i = 0; i < NPK; ++i) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int from = (i * 8 + k) * TPR + t;
            v[i][k] = (adds[0][from] + adds[1][from]) + (adds[2][from] + adds[3][from]);
          }
          const int e = (i * TPR + t) * 8;
          store_piece<false>(out, to + e, dim - e, v[i]);
        }
      }
      __syncthreads();
    };
    add(dw2, 0);
    add(db2, dim);
  }
}

// f(threads per row, pieces a thread) for a row of `dim` elements. WIDE: of a row
// above 8192 elements (backward 4 pieces on 512 threads: the 128 registers that 1024
// threads leave each would not hold a row's three arrays and the two sums).
template <int WIDE, typename F>
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
    f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  } else {
    f(integral_constant<int, WIDE>{}, integral_constant<int, 2048 / WIDE>{});
  }
}

// Blocks that take rows in turn, each with its weights in registers.
constexpr int64_t kForwardBlocks = 4096;

template <bool BI, int RES>
void launch_norm(const LayerNormArgs& a, hipStream_t st) {
  by_width<1024>(a.dim, [&](auto tpr, auto npk) {
    constexpr int TPR = decltype(tpr)::value, NPK = decltype(npk)::value, kBlock = block_threads(TPR);
    const int64_t groups = (a.rows + kBlock / TPR - 1) / (kBlock / TPR);
    const unsigned blocks = static_cast<unsigned>(groups < kForwardBlocks ? groups : kForwardBlocks);
    a.out_bf16 ? layer_norm_kernel<TPR, NPK, BI, RES, true><<<blocks, kBlock, 0, st>>>(a)
               : layer_norm_kernel<TPR, NPK, BI, RES, false><<<blocks, kBlock, 0, st>>>(a);
  });
}

template <bool BI>
void launch_norm_res(const LayerNormArgs& a, hipStream_t st) {
  if (a.residual == nullptr) {
    launch_norm<BI, 0>(a, st);
  } else if (a.res_bf16) {
    launch_norm<BI, 2>(a, st);
  } else {
    launch_norm<BI, 1>(a, st);
  }
}

}  // namespace

int launch_layer_norm(const LayerNormArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  a.in_bf16 ? launch_norm_res<true>(a, st) : launch_norm_res<false>(a, st);
  return static_cast<int>(hipGetLastError());
}

int launch_layer_norm_bwd(const LayerNormBwdArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  int64_t nparts = 0;
  if (a.rows > 0) {
    nparts = layer_norm_bwd_blocks(a.rows, a.dim);
    by_width<512>(a.dim, [&](auto tpr, auto npk) {
      constexpr int TPR = decltype(tpr)::value, NPK = decltype(npk)::value, kBlock = block_threads(TPR);
      const unsigned blocks = static_cast<unsigned>(nparts);
      a.s_bf16 ? layer_norm_bwd_kernel<TPR, NPK, true><<<blocks, kBlock, 0, st>>>(a)
               : layer_norm_bwd_kernel<TPR, NPK, false><<<blocks, kBlock, 0, st>>>(a);
    });
    if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  }
  if (a.dweight != nullptr || a.dbias != nullptr) {
    launch_column_sums(a.workspace, nparts, 2 * a.dim, StoreRows<2>{{a.dweight, a.dbias}, a.dim}, st);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
