// Gated delta rule forward in segments: the states that enter them.
//
// Over a segment the state goes through an affine map of its rows (one per
// column p of the head): s_out[p] = u[p] + s_in[p] F, u [P, N], F [N, N] the same
// for every p. The walk of gated_delta_chunk.h finds both at once: its columns
// are a state from zero with the segment's values, and the N unit vectors
// without any; what they leave is u and F. Here the maps are chained,
//   s_(z+1) = u_z + s_z F_z,
// in order, in float32 matrix instructions (16x16x4): one block of four waves
// per 16 rows of a head's state, a wave a quarter of the N columns; the rows of F
// come straight from memory in the operand's order. The first segment's state is
// copied: h_final may be h0 itself, and the walks of all segments run at once.
// Measured with 16 segments of 8 heads of 128 x 128: 42 us, bound by the chain; the
// next segment's map is in flight while one is applied (when that was built: 50 us,
// 83 without).
#include <hip/hip_runtime.h>

#include "gdr_mma.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kSS = 128 + 4;  // row stride of the state in LDS

template <int NP>
__global__ __launch_bounds__(kThreads) void gdr_join_kernel(const GatedDeltaArgs p, const GdrWork ws, int segs,
                                                            int seg_chunks) {
  __shared__ float sS[16 * kSS];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, m = lane & 15, g = lane >> 4;
  const int N = static_cast<int>(p.dstate), P = static_cast<int>(p.headdim), H = static_cast<int>(p.nheads);
  const int groups = (P + 15) / 16;
  const int place = gdr_xcd_place(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), groups);
  const int bh = place / groups, p0 = place % groups * 16;
  const int64_t len = gdr_row_steps(p.seqlens, bh / H, p.seqlen);
  const int64_t most = static_cast<int64_t>(seg_chunks) * kGdrC;
  const float* maps = ws.map + static_cast<int64_t>(bh) * segs * (P + N) * N;
  for (int i = tid; i < 16 * kSS; i += kThreads) sS[i] = 0.0f;
  const int64_t at0 = (static_cast<int64_t>(bh) * P + p0) * N;
  const int mine = (P - p0 < 16 ? P - p0 : 16) * N;
  for (int i = tid; i < mine; i += kThreads) ws.seg[at0 + i] = p.h0 != nullptr ? p.h0[at0 + i] : 0.0f;
  __syncthreads();
  // Tile t of the wave: column m is n = 32 w + 16 t + m; element i is row p0 + 4 g
  // + i. Rows and columns past P and N are read as the last ones (no load in a
  // branch): what they give is not kept, and the state's columns past N are 0.
  const int64_t map = static_cast<int64_t>(P + N) * N;
  const int n0 = 32 * w + m < N ? 32 * w + m : N - 1, n1 = 32 * w + 16 + m < N ? 32 * w + 16 + m : N - 1;
  float f0[NP / 4], f1[NP / 4], u[2][4];
  const auto fetch = [&](int z) __attribute__((always_inline)) {
    const float* at = maps + z * map;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = p0 + 4 * g + i < P ? p0 + 4 * g + i : P - 1;
      u[0][i] = at[static_cast<int64_t>(row) * N + n0];
      u[1][i] = at[static_cast<int64_t>(row) * N + n1];
    }
    at += static_cast<int64_t>(P) * N;
#pragma unroll
    for (int k = 0; k < NP; k += 4) {
      const float* row = at + (k + g < N ? k + g : N - 1) * N;
      f0[k / 4] = row[n0];
      f1[k / 4] = row[n1];
    }
  };
  int last = 0;  // maps of segments 0 .. last - 1 are there
  for (int z = 0; z + 1 < segs && len > (z + 1) * most; ++z) last = z + 1;
  if (last == 0) return;
  fetch(0);
  for (int z = 0; z < last; ++z) {
    f32x4_t acc[2];
    float b0[NP / 4], b1[NP / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[0][i] = u[0][i], acc[1][i] = u[1][i];
#pragma unroll
    for (int k = 0; k < NP / 4; ++k) b0[k] = f0[k], b1[k] = f1[k];
    fetch(z + 1 < last ? z + 1 : z);  // the next segment's, while this one's is worked on
    if (z > 0) {  // (the first segment's walk started from the state itself)
#pragma unroll
      for (int k = 0; k < NP; k += 4) {
        const float a = sS[m * kSS + k + g];
        acc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, b0[k / 4], acc[0], 0, 0, 0);
        acc[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, b1[k / 4], acc[1], 0, 0, 0);
      }
    }
    __syncthreads();
    float* out = ws.seg + (z + 1) * ws.seg_stride + at0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = 32 * w + 16 * t + m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * g + i;
        sS[row * kSS + n] = n < N ? acc[t][i] : 0.0f;
        if (p0 + row < P && n < N) out[static_cast<int64_t>(row) * N + n] = acc[t][i];
      }
    }
    __syncthreads();
  }
}

}  // namespace

void launch_gdr_join(const GatedDeltaArgs& a, const GdrWork& ws, int segs, int seg_chunks, hipStream_t st) {
  const unsigned blocks = static_cast<unsigned>(a.batch * a.nheads * ((a.headdim + 15) / 16));
  if (a.dstate <= 64) {
    gdr_join_kernel<64><<<blocks, kThreads, 0, st>>>(a, ws, segs, seg_chunks);
  } else {
    gdr_join_kernel<128><<<blocks, kThreads, 0, st>>>(a, ws, segs, seg_chunks);
  }
}

}  // namespace ssm
