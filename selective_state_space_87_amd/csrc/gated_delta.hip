// Gated delta rule, step by step: the single-token update, and the forward of
// the shortest sequences; and the choice between this and the chunked form.
//
// Per (batch row, head), with the state S [N, P] and a = exp(dt A), beta:
//   S <- a S;  e = beta (v - k^T S);  S <- S + k e^T;  y = scale q^T S
// The columns of S (one per channel p) do not touch each other, so a column is
// the unit of work. Both readouts are taken of the state before the write and
// corrected by a scalar, so that a step passes over its state once:
//   k^T (a S) = a (k . s_p),   q^T S_new = a (q . s_p) + e_p (q . k)
//
// Mapping. Eight lanes own a column (lane j of them holds n = 32 i + 4 j + 0..3,
// so that the eight read 128 consecutive bytes of a state row), a wave eight
// columns, a block of four waves 32. The sums over n are three DPP adds inside
// the eight lanes; no LDS and no barrier. q and k are read by every group of
// eight lanes (from L1 after the first), and their norms come out of the same
// sums.
//
// The update is bound by HBM: the state is read and written once. 128 batch rows
// of 32 heads of 128 x 128 (537 MB): 109 us, 4.9 TB/s, 117 us the call, as fast as a large copy.
#include <hip/hip_runtime.h>

#include "device_math.h"
#include "gated_delta.h"
#include "gdr_mma.h"

namespace ssm {

namespace {

constexpr int kRecThreads = 256;
constexpr int kRecCols = kRecThreads / 8;

// Four consecutive elements n .. n+3 of a row (zeros past `count`).
template <bool BF16, bool VEC>
__device__ __forceinline__ void load4(const void* base, int64_t at, int n, int count, float (&out)[4]) {
  if constexpr (VEC) {
    if (n < count) {  // count is a multiple of 4
      if constexpr (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at + n);
        out[0] = __uint_as_float(w.x << 16);
        out[1] = __uint_as_float(w.x & 0xffff0000u);
        out[2] = __uint_as_float(w.y << 16);
        out[3] = __uint_as_float(w.y & 0xffff0000u);
      } else {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + n);
        out[0] = w.x;
        out[1] = w.y;
        out[2] = w.z;
        out[3] = w.w;
      }
    } else {
      out[0] = out[1] = out[2] = out[3] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = n + i < count ? load_elem<BF16>(base, at + n + i) : 0.0f;
  }
}

// Sum over the eight lanes of a column, the same in all of them.
__device__ __forceinline__ float sum8(float v) {
  v += quad_xor<1>(v);
  v += quad_xor<2>(v);
  return v + dpp_f<0x141>(v);  // row_half_mirror: the other quad of the eight
}

template <int NC, bool BF16_IN, bool BF16_OUT, bool VEC>
__global__ __launch_bounds__(kRecThreads) void gdr_recurrent_kernel(const GatedDeltaArgs p) {
  const int tid = threadIdx.x, j = tid & 7;
  const int N = static_cast<int>(p.dstate), P = static_cast<int>(p.headdim);
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads);
  const int pblocks = (P + kRecCols - 1) / kRecCols;
  const int item = static_cast<int>(blockIdx.x) / pblocks;
  const int b = item / H, h = item % H, g = h / (H / G);
  const int col = (static_cast<int>(blockIdx.x) % pblocks) * kRecCols + (tid >> 3);
  const bool on = col < P;
  const int64_t L = p.seqlen;
  const int64_t len = gdr_row_steps(p.seqlens, b, L);
  const int64_t row0 = static_cast<int64_t>(b) * L;
  const int64_t sb = (static_cast<int64_t>(item) * P + (on ? col : 0)) * N;

  float s[NC][4];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (p.h0 != nullptr && on) {
      load4<false, VEC>(p.h0, sb, 32 * i + 4 * j, N, s[i]);
    } else {
      s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
    }
  }
  const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;

  for (int64_t t = 0; t < len; ++t) {
    const int64_t row = row0 + t;
    float q[NC][4], k[NC][4];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      load4<BF16_IN, VEC>(p.q, row * p.q_step + static_cast<int64_t>(g) * N, 32 * i + 4 * j, N, q[i]);
      load4<BF16_IN, VEC>(p.k, row * p.k_step + static_cast<int64_t>(g) * N, 32 * i + 4 * j, N, k[i]);
    }
    const float v = on ? load_elem<BF16_IN>(p.v, row * p.v_step + static_cast<int64_t>(h) * P + col) : 0.0f;
    const float a = exp2_hw(gdr_log_decay(p, load_elem<BF16_IN>(p.dt, row * H + h), bias, A) * kLog2e);
    const float beta = gdr_beta(p, load_elem<BF16_IN>(p.beta, row * H + h));
    float qq = 0.0f, kk = 0.0f, qk = 0.0f, qs = 0.0f, ks = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qq = fmaf(q[i][e], q[i][e], qq);
        kk = fmaf(k[i][e], k[i][e], kk);
        qk = fmaf(q[i][e], k[i][e], qk);
        qs = fmaf(q[i][e], s[i][e], qs);
        ks = fmaf(k[i][e], s[i][e], ks);
      }
    }
    qk = sum8(qk);
    qs = sum8(qs);
    ks = sum8(ks);
    float rq = 1.0f, rk = 1.0f;
    if (p.qk_l2norm) {
      rq = rsqrtf(sum8(qq) + kL2NormEps);
      rk = rsqrtf(sum8(kk) + kL2NormEps);
    }
    const float e = beta * fmaf(-a * rk, ks, v);
    const float w = e * rk;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
      for (int n = 0; n < 4; ++n) s[i][n] = fmaf(k[i][n], w, a * s[i][n]);
    }
    const float y = p.scale * rq * fmaf(a, qs, w * qk);
    if (on && j == 0) store_elem<BF16_OUT>(p.y, (row * H + h) * P + col, y);
  }
  for (int64_t t = len; t < L; ++t) {
    if (on && j == 0) store_elem<BF16_OUT>(p.y, ((row0 + t) * H + h) * P + col, 0.0f);
  }
  if (p.h_final != nullptr && on) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int n = 32 * i + 4 * j;
      if constexpr (VEC) {
        if (n < N) {
          *reinterpret_cast<float4*>(p.h_final + sb + n) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (n + e < N) p.h_final[sb + n + e] = s[i][e];
        }
      }
    }
  }
}

bool on_boundary(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <int NC, bool BI, bool BO>
void launch_rec(const GatedDeltaArgs& a, bool vec, unsigned blocks, hipStream_t st) {
  if (vec) {
    gdr_recurrent_kernel<NC, BI, BO, true><<<blocks, kRecThreads, 0, st>>>(a);
  } else {
    gdr_recurrent_kernel<NC, BI, BO, false><<<blocks, kRecThreads, 0, st>>>(a);
  }
}

template <int NC>
void launch_rec_types(const GatedDeltaArgs& a, bool vec, unsigned blocks, hipStream_t st) {
  if (a.in_bf16) {
    a.out_bf16 ? launch_rec<NC, true, true>(a, vec, blocks, st) : launch_rec<NC, true, false>(a, vec, blocks, st);
  } else {
    a.out_bf16 ? launch_rec<NC, false, true>(a, vec, blocks, st) : launch_rec<NC, false, false>(a, vec, blocks, st);
  }
}

}  // namespace

int launch_gated_delta_recurrent(const GatedDeltaArgs& a, void* stream) {
  const uintptr_t eb = a.in_bf16 ? 8 : 16;
  const bool vec = a.dstate % 4 == 0 && a.q_step % 4 == 0 && a.k_step % 4 == 0 && on_boundary(a.q, eb) &&
                   on_boundary(a.k, eb) && on_boundary(a.h0, 16) && on_boundary(a.h_final, 16);
  const unsigned blocks =
      static_cast<unsigned>(a.batch * a.nheads * ((a.headdim + kRecCols - 1) / kRecCols));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.dstate <= 32) {
    launch_rec_types<1>(a, vec, blocks, st);
  } else if (a.dstate <= 64) {
    launch_rec_types<2>(a, vec, blocks, st);
  } else {
    launch_rec_types<4>(a, vec, blocks, st);
  }
  return static_cast<int>(hipGetLastError());
}

int launch_gated_delta_update(const GatedDeltaArgs& a, void* stream) {
  return launch_gated_delta_recurrent(a, stream);
}

namespace {

GdrWork gdr_work(void* workspace, const GdrPlan& pl, const GatedDeltaArgs& a) {
  char* base = static_cast<char*>(workspace);
  GdrWork ws{};
  ws.T = reinterpret_cast<_Float16*>(base + pl.off_t);
  ws.Pm = reinterpret_cast<_Float16*>(base + pl.off_p);
  ws.K = reinterpret_cast<_Float16*>(base + pl.off_k);
  ws.Q = reinterpret_cast<_Float16*>(base + pl.off_q);
  ws.fac = reinterpret_cast<float*>(base + pl.off_fac);
  ws.Tt = reinterpret_cast<_Float16*>(base + pl.off_tt);
  ws.Pt = ws.Pm;
  ws.S = reinterpret_cast<float*>(base + pl.off_s);
  ws.X = reinterpret_cast<float*>(base + pl.off_x);
  ws.E = reinterpret_cast<float*>(base + pl.off_e);
  ws.top = reinterpret_cast<float*>(base + pl.off_top);
  ws.part = reinterpret_cast<double*>(base + pl.off_part);
  ws.map = reinterpret_cast<float*>(base + pl.off_map);
  ws.seg = reinterpret_cast<float*>(base + pl.off_seg);
  ws.seg_stride = a.batch * a.nheads * a.headdim * a.dstate;
  return ws;
}

bool rows_on_16(const GatedDeltaArgs& a) {
  const int64_t per16 = a.in_bf16 ? 8 : 4;  // elements in 16 bytes
  return a.dstate % 8 == 0 && a.q_step % per16 == 0 && a.k_step % per16 == 0 && on_boundary(a.q, 16) &&
         on_boundary(a.k, 16);
}

int launch_chunks(const GatedDeltaArgs& a, const GdrWork& ws, const GdrPlan& pl, bool backward, void* stream) {
  if (const int e = launch_gdr_prep(a, ws, pl.chunks, backward, rows_on_16(a), stream)) return e;
  if (backward && gdr_both_at_once(a)) return 0;  // (walked by launch_gdr_reverse)
  return a.in_bf16 ? launch_gdr_chunk_b(a, ws, pl, backward, stream)
                   : launch_gdr_chunk_f(a, ws, pl, backward, stream);
}

}  // namespace

int launch_gated_delta(const GatedDeltaArgs& a, void* stream) {
  const GdrPlan pl = plan_gated_delta(a.batch, a.seqlen, a.nkheads, a.nheads, a.headdim, a.dstate, a.in_bf16, false);
  if (pl.recurrent) return launch_gated_delta_recurrent(a, stream);
  return launch_chunks(a, gdr_work(a.workspace, pl, a), pl, false, stream);
}

int launch_gated_delta_bwd(const GatedDeltaBwdArgs& a, void* stream) {
  const GatedDeltaArgs& f = a.f;
  const GdrPlan pl = plan_gated_delta(f.batch, f.seqlen, f.nkheads, f.nheads, f.headdim, f.dstate, f.in_bf16, true);
  const GdrWork ws = gdr_work(f.workspace, pl, f);
  if (pl.chunks > 0 && f.batch > 0) {
    if (const int e = launch_chunks(f, ws, pl, true, stream)) return e;
  }
  if (f.batch > 0) {
    if (const int e = launch_gdr_reverse(a, ws, pl.chunks, stream)) return e;
  }
  return launch_gdr_grads(a, ws, f.batch > 0 ? pl.chunks : 0, stream);
}

}  // namespace ssm
