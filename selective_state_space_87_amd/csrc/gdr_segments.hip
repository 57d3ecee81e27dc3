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
  const int bh = static_cast<int>(blockIdx.x) / groups, p0 = (static_cast<int>(blockIdx.x) % groups) * 16;
  const int64_t len = gdr_row_steps(p.seqlens, bh / H, p.seqlen);
  const int64_t most = static_cast<int64_t>(seg_chunks) * kGdrC;
  const float* maps = ws.map + static_cast<int64_t>(bh) * segs * (P + N) * N;
  for (int i = tid; i < 16 * kSS; i += kThreads) sS[i] = 0.0f;
  const int64_t at0 = (static_cast<int64_t>(bh) * P + p0) * N;
  const int mine = (P - p0 < 16 ? P - p0 : 16) * N;
  for (int i = tid; i < mine; i += kThreads) ws.seg[at0 + i] = p.h0 != nullptr ? p.h0[at0 + i] : 0.0f;
  __syncthreads();
  // Tile u of the wave: column m is n = 32 w + 16 u + m; element i is row p0 + 4 g + i.
  for (int z = 0; z + 1 < segs && len > (z + 1) * most; ++z) {
    const float* u = maps + static_cast<int64_t>(z) * (P + N) * N;
    const float* F = u + static_cast<int64_t>(P) * N;
    f32x4_t acc[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = 32 * w + 16 * t + m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = p0 + 4 * g + i;
        acc[t][i] = row < P && n < N ? u[static_cast<int64_t>(row) * N + n] : 0.0f;
      }
    }
    if (z > 0) {  // (the first segment's walk started from the state itself)
      // past N the state's columns in LDS are 0: rows and columns of F past it
      // may be any, the last ones here (no load in a branch)
      const int n0 = 32 * w + m < N ? 32 * w + m : N - 1, n1 = 32 * w + 16 + m < N ? 32 * w + 16 + m : N - 1;
      float b0[NP / 4], b1[NP / 4];  // all of them in flight at once
#pragma unroll
      for (int k = 0; k < NP; k += 4) {
        const float* row = F + (k + g < N ? k + g : N - 1) * N;
        b0[k / 4] = row[n0];
        b1[k / 4] = row[n1];
      }
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
