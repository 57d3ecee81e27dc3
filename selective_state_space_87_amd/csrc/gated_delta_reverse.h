// Gated delta rule backward, the walk back over a head's chunks (see gdr_mma.h).
// With the gradient X of the state leaving a chunk, dY the output's:
//   G  = Pm^T dY + diag(w) K X            (of E, as the later ones see it)
//   dE = T^T G                            (of V - diag(e^c) K S; also dV)
//   X' = e^(c_end) X + Q^T (qf dY) - K^T (kf dE)
// the mirror image of the forward's walk: a wave owns 16 columns of X in
// registers, and the chain of products stays inside it. X is left in the
// workspace for every chunk (the gradient of its leaving state), dE in dv.
#pragma once

#include "gdr_mma.h"

namespace ssm {

template <int NP, bool BF16, bool VEC, int NW>
struct GdrBack {
  static constexpr int NT = 64 * NW;
  static constexpr int RAW = BF16 ? 1 : 2;
  static constexpr int RS = NP + 8;
  static constexpr int kMat = RAW * kGdrC * RS;
  static constexpr int kTri = kGdrPieceHalves;
  static constexpr int kFac = 5 * kGdrC + 4;            // K, Q, W, Tt, P factors and the end's
  static constexpr int kBufBytes = (2 * kMat + 2 * kTri) * 2 + kFac * 4;
  static constexpr int NBUF = 2 * kBufBytes <= 160 * 1024 ? 2 : 1;
  static constexpr int NKQ = kGdrC * NP / 8 / NT;
  static constexpr int NTL = kTri / 8 / NT;
  static constexpr int NFL = (5 * kGdrC + NT - 1) / NT;
};

template <int NP, bool BF16, bool VEC, int NW>
__global__ __launch_bounds__(64 * NW) void gdr_reverse_kernel(const GatedDeltaBwdArgs a, const GdrWork ws, int chunks) {
  using W = GdrBack<NP, BF16, VEC, NW>;
  constexpr int NT = W::NT, RAW = W::RAW, RS = W::RS, NJ = NP / 16, NK = NP / 32;
  constexpr int EB = BF16 ? 2 : 4;
  __shared__ __align__(16) char lds[W::NBUF][W::kBufBytes];
  const GatedDeltaArgs& p = a.f;

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, m = lane & 15, g = lane >> 4;
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads);
  const int N = static_cast<int>(p.dstate), P = static_cast<int>(p.headdim);
  const int pblocks = (P + 16 * NW - 1) / (16 * NW);
  const int bh = static_cast<int>(blockIdx.x) / pblocks;
  const int b = bh / H, h = bh % H, kh = h / (H / G);
  const int col = (static_cast<int>(blockIdx.x) % pblocks) * 16 * NW + 16 * w + m;
  const bool col_ok = col < P;
  const int64_t L = p.seqlen;
  const int64_t len = gdr_row_steps(p.seqlens, b, L);
  const int n_chunks = static_cast<int>((len + kGdrC - 1) / kGdrC);
  const int64_t row_b = static_cast<int64_t>(b) * L;
  const int64_t item0 = static_cast<int64_t>(bh) * chunks;
  const int64_t sb = (static_cast<int64_t>(bh) * P + (col_ok ? col : 0)) * N;
  const uint32_t yrow = static_cast<uint32_t>(H * P);

  f32x4_t X[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
      X[j][i] = (a.dh_final != nullptr && col_ok && n < N) ? a.dh_final[sb + n] : 0.0f;
    }
  }

  Raw8<BF16, VEC> kr[W::NKQ], qr[W::NKQ];
  float ku[W::NKQ], qu[W::NKQ], fr[W::NFL], fend = 0.0f;
  u32x4_t tr[W::NTL], pr[W::NTL];
  float yr[16];

  const auto factor = [](int i) { return i == 3 ? static_cast<int>(kFacTt) : (i == 4 ? static_cast<int>(kFacP) : kFacK + i); };
  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
    const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
    const int64_t row0 = row_b + t0;
    const uint32_t ks = static_cast<uint32_t>(p.k_step), qs = static_cast<uint32_t>(p.q_step);
    const rsrc_t rk = rows_buffer<EB>(p.k, row0 * p.k_step + static_cast<int64_t>(kh) * N, rows, ks, N);
    const rsrc_t rq = rows_buffer<EB>(p.q, row0 * p.q_step + static_cast<int64_t>(kh) * N, rows, qs, N);
    const rsrc_t ry = rows_buffer<4>(a.dy, row0 * yrow + static_cast<int64_t>(h) * P, rows, yrow, P);
    const float* fac = ws.fac + (item0 + c) * (kGdrFactors * kGdrC);
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      const int e = (i * NT + tid) * 8, t = e / NP, n = e % NP;
      kr[i] = load_raw8<BF16, VEC>(rk, t, n, ks, N);
      qr[i] = load_raw8<BF16, VEC>(rq, t, n, qs, N);
      ku[i] = fac[kFacKup * kGdrC + t];
      qu[i] = fac[kFacQup * kGdrC + t];
    }
    const u32x4_t* T = reinterpret_cast<const u32x4_t*>(ws.Tt + (item0 + c) * kGdrPieceHalves);
    const u32x4_t* Pt = reinterpret_cast<const u32x4_t*>(ws.Pt + (item0 + c) * kGdrPieceHalves);
#pragma unroll
    for (int i = 0; i < W::NTL; ++i) {
      tr[i] = T[i * NT + tid];
      pr[i] = Pt[i * NT + tid];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * NT + tid;
      fr[i] = fac[factor(e / kGdrC % 5) * kGdrC + e % kGdrC];
    }
    fend = fac[kFacEnd * kGdrC];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t off = (static_cast<uint32_t>(16 * tt + 4 * g + i) * yrow + static_cast<uint32_t>(col)) * 4;
        yr[4 * tt + i] = __uint_as_float(buffer_load_bits<false>(ry, col_ok ? off : kOutOfRange));
      }
    }
  };
  auto stage = [&](int buf) __attribute__((always_inline)) {
    _Float16* sK = reinterpret_cast<_Float16*>(lds[buf]);
    _Float16* sQ = sK + W::kMat;
    u32x4_t* sT = reinterpret_cast<u32x4_t*>(sQ + W::kMat);
    u32x4_t* sP = sT + W::kTri / 8;
    float* sF = reinterpret_cast<float*>(sP + W::kTri / 8);
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      const int e = (i * NT + tid) * 8, t = e / NP, n = e % NP;
      float x[8];
      raw8_values<BF16, VEC>(kr[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= ku[i];
      half8_t hi = halves(x);
      *reinterpret_cast<half8_t*>(sK + t * RS + n) = hi;
      if constexpr (RAW == 2) *reinterpret_cast<half8_t*>(sK + kGdrC * RS + t * RS + n) = rest(x, hi);
      raw8_values<BF16, VEC>(qr[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= qu[i];
      hi = halves(x);
      *reinterpret_cast<half8_t*>(sQ + t * RS + n) = hi;
      if constexpr (RAW == 2) *reinterpret_cast<half8_t*>(sQ + kGdrC * RS + t * RS + n) = rest(x, hi);
    }
#pragma unroll
    for (int i = 0; i < W::NTL; ++i) {
      sT[i * NT + tid] = tr[i];
      sP[i * NT + tid] = pr[i];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * NT + tid;
      if (e < 5 * kGdrC) sF[e] = fr[i];
    }
    if (tid == 0) sF[5 * kGdrC] = fend;
  };

  if (n_chunks > 0) {
    fetch(n_chunks - 1);
    stage(0);
  }
  __syncthreads();

  for (int step = 0; step < n_chunks; ++step) {
    const int c = n_chunks - 1 - step;
    const int buf = W::NBUF == 2 ? (step & 1) : 0;
    const _Float16* sK = reinterpret_cast<const _Float16*>(lds[buf]);
    const _Float16* sQ = sK + W::kMat;
    const _Float16* sT = sQ + W::kMat;
    const _Float16* sP = sT + W::kTri;
    const float* sF = reinterpret_cast<const float*>(sP + W::kTri);
    f32x4_t Y[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) Y[i / 4][i % 4] = yr[i];
    fetch(c > 0 ? c - 1 : 0);  // (in no branch: a conditional load is waited for where the branches join)

    const int64_t item = item0 + c;
    {
      if (col_ok) {
        float* dst = ws.X + (item * P + col) * N;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int n = 32 * (j / 2) + 8 * g + 4 * (j & 1);
          if (N % 4 == 0) {
            if (n < N) *reinterpret_cast<f32x4_t*>(dst + n) = X[j];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (n + i < N) dst[n + i] = X[j][i];
            }
          }
        }
      }
    }
    const float xtop = tiles_absmax<NJ>(X), ytop = tiles_absmax<4>(Y);
    const Pow2 sx = pow2_to_top(xtop), sy = pow2_to_top(ytop);

    // G = Pm^T dY + diag(w) K X
    f32x4_t D[4];
    {
      half8_t Xh[NK], Xl[NK], Yh[2], Yl[2];
#pragma unroll
      for (int q = 0; q < NK; ++q) tiles_to_operand<true>(X[2 * q], X[2 * q + 1], sx.up, Xh[q], Xl[q]);
#pragma unroll
      for (int q = 0; q < 2; ++q) tiles_to_operand<true>(Y[2 * q], Y[2 * q + 1], sy.up, Yh[q], Yl[q]);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        f32x4_t kx = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, py = kx;
#pragma unroll
        for (int q = 0; q < NK; ++q) {
          const int at = (16 * tt + m) * RS + 32 * q + 8 * g;
          const half8_t k = *reinterpret_cast<const half8_t*>(sK + at);
          kx = mfma16(k, Xh[q], kx);
          kx = mfma16(k, Xl[q], kx);
          if constexpr (RAW == 2) kx = mfma16(*reinterpret_cast<const half8_t*>(sK + kGdrC * RS + at), Xh[q], kx);
        }
#pragma unroll
        for (int q = tt / 2; q < 2; ++q) {
          const _Float16* at = sP + gdr_frag_up(tt, q) * 2 * kGdrFragHalves + lane * 8;
          const half8_t hi = *reinterpret_cast<const half8_t*>(at);
          py = mfma16(hi, Yh[q], py);
          py = mfma16(hi, Yl[q], py);
          py = mfma16(*reinterpret_cast<const half8_t*>(at + kGdrFragHalves), Yh[q], py);
        }
        const f32x4_t fw = *reinterpret_cast<const f32x4_t*>(sF + 2 * kGdrC + 16 * tt + 4 * g);
        const f32x4_t fp = *reinterpret_cast<const f32x4_t*>(sF + 4 * kGdrC + 16 * tt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) D[tt][i] = fmaf(fw[i] * sx.down, kx[i], fp[i] * sy.down * py[i]);
      }
    }
    // dE = T^T G
    f32x4_t E[4];
    {
      const Pow2 sd = pow2_to_top(tiles_absmax<4>(D));
      half8_t Dh[2], Dl[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) tiles_to_operand<true>(D[2 * q], D[2 * q + 1], sd.up, Dh[q], Dl[q]);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        E[tt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = tt / 2; q < 2; ++q) {
          const _Float16* at = sT + gdr_frag_up(tt, q) * 2 * kGdrFragHalves + lane * 8;
          const half8_t hi = *reinterpret_cast<const half8_t*>(at);
          E[tt] = mfma16(hi, Dh[q], E[tt]);
          E[tt] = mfma16(hi, Dl[q], E[tt]);
          E[tt] = mfma16(*reinterpret_cast<const half8_t*>(at + kGdrFragHalves), Dh[q], E[tt]);
        }
        const f32x4_t f = *reinterpret_cast<const f32x4_t*>(sF + 3 * kGdrC + 16 * tt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) E[tt][i] *= f[i] * sd.down;
      }
    }
    const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
    const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
    const int out_rows = static_cast<int>(L - t0 < kGdrC ? L - t0 : kGdrC);
    const rsrc_t rv = rows_buffer<4>(a.dv, (row_b + t0) * yrow + static_cast<int64_t>(h) * P, out_rows, yrow, P);
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * tt + 4 * g + i;
        const uint32_t off = (static_cast<uint32_t>(t) * yrow + static_cast<uint32_t>(col)) * 4;
        buffer_store_f32<false>(t < rows ? E[tt][i] : 0.0f, rv, col_ok ? off : kOutOfRange);
      }
    }
    const float etop = tiles_absmax<4>(E);
    {
      const float mx = lanes16_max(xtop), my = lanes16_max(ytop), me = lanes16_max(etop);
      if (lane == 0 && col < P) {
        float* top = ws.top + item * kGdrMaxima * kGdrMaxSlots + col / 16 * 2;
        top[kMaxX * kGdrMaxSlots] = top[kMaxX * kGdrMaxSlots + 1] = mx;
        top[kMaxDY * kGdrMaxSlots] = top[kMaxDY * kGdrMaxSlots + 1] = my;
        top[kMaxDE * kGdrMaxSlots] = top[kMaxDE * kGdrMaxSlots + 1] = me;
      }
    }
    // X' = e^(c_end) X + Q^T (qf dY) - K^T (kf dE)
    {
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const f32x4_t fk = *reinterpret_cast<const f32x4_t*>(sF + 0 * kGdrC + 16 * tt + 4 * g);
        const f32x4_t fq = *reinterpret_cast<const f32x4_t*>(sF + 1 * kGdrC + 16 * tt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          Y[tt][i] *= fq[i];
          E[tt][i] *= -fk[i];
        }
      }
      // one scale for both, so that one accumulator takes them
      const Pow2 s = pow2_to_top(fmaxf(tiles_absmax<4>(Y), tiles_absmax<4>(E)));
      half8_t Yh[2], Yl[2], Eh[2], El[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        tiles_to_operand<true>(Y[2 * q], Y[2 * q + 1], s.up, Yh[q], Yl[q]);
        tiles_to_operand<true>(E[2 * q], E[2 * q + 1], s.up, Eh[q], El[q]);
      }
      const float end = sF[5 * kGdrC];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int at = (32 * q + 4 * g + (m >> 2)) * RS + 32 * (j / 2) + 8 * (m & 3) + 4 * (j & 1);
          const auto column = [&](const _Float16* mat) __attribute__((always_inline)) {
            return __builtin_shufflevector(lds_column4(mat + at), lds_column4(mat + at + 16 * RS), 0, 1, 2, 3, 4, 5, 6, 7);
          };
          const half8_t kc = column(sK), qc = column(sQ);
          acc = mfma16(qc, Yh[q], acc);
          acc = mfma16(qc, Yl[q], acc);
          acc = mfma16(kc, Eh[q], acc);
          acc = mfma16(kc, El[q], acc);
          if constexpr (RAW == 2) {
            acc = mfma16(column(sQ + kGdrC * RS), Yh[q], acc);
            acc = mfma16(column(sK + kGdrC * RS), Eh[q], acc);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) X[j][i] = fmaf(acc[i], s.down, end * X[j][i]);
      }
    }

    if constexpr (W::NBUF == 1) __syncthreads();
    if (step + 1 < n_chunks) stage(W::NBUF == 2 ? ((step + 1) & 1) : 0);
    __syncthreads();
  }

  for (int64_t t = static_cast<int64_t>(n_chunks) * kGdrC + g; t < L; t += 4) {
    if (col_ok) a.dv[(row_b + t) * yrow + static_cast<int64_t>(h) * P + col] = 0.0f;
  }
  if (a.dh0 != nullptr && col_ok) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
        if (n < N) a.dh0[sb + n] = X[j][i];
      }
    }
  }
}

template <int NP, bool BF16, bool VEC>
void gdr_launch_reverse_nw(const GatedDeltaBwdArgs& a, const GdrWork& ws, int chunks, hipStream_t st) {
  const int64_t bh = a.f.batch * a.f.nheads;
  const int64_t slices = (a.f.headdim + 15) / 16;
  if (slices <= 2) {
    gdr_reverse_kernel<NP, BF16, VEC, 2><<<static_cast<unsigned>(bh * ((slices + 1) / 2)), 128, 0, st>>>(a, ws, chunks);
  } else {
    gdr_reverse_kernel<NP, BF16, VEC, 4><<<static_cast<unsigned>(bh * ((slices + 3) / 4)), 256, 0, st>>>(a, ws, chunks);
  }
}

}  // namespace ssm
