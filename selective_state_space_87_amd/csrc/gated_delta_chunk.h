// Gated delta rule, the walk over a head's chunks (see gdr_mma.h for the
// chunk's equations, operand halves and layouts). Included by one source file
// per input type.
//
// A wave owns 16 columns of a head's state [N, P] and keeps them in registers,
// as the accumulators of the state's update and, split into halves, as the
// operand of K S and Q S. A chunk is a chain of five products inside the wave:
//   K S, Q S  ->  E = T (V - ..)  ->  Y = .. + Pm E,  S' = .. + K^T (w E)
// with no exchange between waves. A block of NW waves (16 NW columns) shares
// K, Q (halves made while staging), T, Pm and the factors through LDS; the next chunk's are in
// flight in registers meanwhile, and go into the other LDS buffer where two
// fit (one barrier a chunk) or into the same one (two barriers).
#pragma once

#include "gdr_mma.h"

namespace ssm {

// KEEP: the backward's pass over the chunks, which leaves the entering states
// and E in the workspace and no y (neither Q nor Pm is touched).
template <int NP, bool BF16, bool OB16, bool VEC, int NW, bool KEEP>
struct GdrWalk {
  static constexpr int NT = 64 * NW;
  static constexpr int RAW = BF16 ? 1 : 2;
  static constexpr int OP = OB16 ? 1 : 2;               // halves in the products that only y sees
  static constexpr int RS = NP + 8;                     // row stride of K and Q in LDS (halves)
  static constexpr int kMat = RAW * kGdrC * RS;         // halves of K (or Q)
  static constexpr int kT = kGdrFrags * 2 * kGdrFragHalves;
  static constexpr int kP = KEEP ? 0 : kGdrFrags * OP * kGdrFragHalves;
  static constexpr int kFac = 5 * kGdrC + 4;            // K, Q, W, T, P factors and the end's
  static constexpr int kBufBytes = ((KEEP ? 1 : 2) * kMat + kT + kP) * 2 + kFac * 4;
  static constexpr int NBUF = 2 * kBufBytes <= 160 * 1024 ? 2 : 1;
  static constexpr int NKQ = kGdrC * NP / 8 / NT;       // 8-element pieces of K (and Q) a thread
  static constexpr int NTL = (kT / 8 + NT - 1) / NT;    // 16-byte pieces of T a thread
  static constexpr int NPL = (kP / 8 + NT - 1) / NT;
  static constexpr int NFL = (5 * kGdrC + NT - 1) / NT;
};

template <int NP, bool BF16, bool OB16, bool VEC, int NW, bool KEEP>
__global__ __launch_bounds__(64 * NW) void gdr_chunk_kernel(const GatedDeltaArgs p, const GdrWork ws, int chunks) {
  using W = GdrWalk<NP, BF16, OB16, VEC, NW, KEEP>;
  constexpr int NT = W::NT, RAW = W::RAW, OP = W::OP, RS = W::RS, NJ = NP / 16, NK = NP / 32;
  constexpr int EB = BF16 ? 2 : 4;
  __shared__ __align__(16) char lds[W::NBUF][W::kBufBytes];

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

  // The state: tile j = 2 q + u, element i is n = 32 q + 8 g + 4 u + i of
  // column `col`, so that tiles 2 q and 2 q + 1 together are n = 32 q + 8 g + 0..7:
  // the contraction order in which a lane's piece of a K row is contiguous.
  f32x4_t S[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
      S[j][i] = (p.h0 != nullptr && col_ok && n < N) ? p.h0[sb + n] : 0.0f;
    }
  }

  Raw8<BF16, VEC> kr[W::NKQ], qr[W::NKQ];
  float ku[W::NKQ], qu[W::NKQ], fr[W::NFL], fend = 0.0f;
  u32x4_t tr[W::NTL], pr[W::NPL > 0 ? W::NPL : 1];
  storage_t<BF16> vr[16];

  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
    const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
    const int64_t row0 = row_b + t0;
    const uint32_t ks = static_cast<uint32_t>(p.k_step), qs = static_cast<uint32_t>(p.q_step);
    const uint32_t vs = static_cast<uint32_t>(p.v_step);
    const rsrc_t rk = rows_buffer<EB>(p.k, row0 * p.k_step + static_cast<int64_t>(kh) * N, rows, ks, N);
    const rsrc_t rq = rows_buffer<EB>(p.q, row0 * p.q_step + static_cast<int64_t>(kh) * N, rows, qs, N);
    const rsrc_t rv = rows_buffer<EB>(p.v, row0 * p.v_step + static_cast<int64_t>(h) * P, rows, vs, P);
    const float* fac = ws.fac + (item0 + c) * (kGdrFactors * kGdrC);
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      const int e = (i * NT + tid) * 8, t = e / NP, n = e % NP;
      kr[i] = load_raw8<BF16, VEC>(rk, t, n, ks, N);
      if constexpr (!KEEP) qr[i] = load_raw8<BF16, VEC>(rq, t, n, qs, N);
      ku[i] = fac[kFacKup * kGdrC + t];
      if constexpr (!KEEP) qu[i] = fac[kFacQup * kGdrC + t];
    }
    const u32x4_t* T = reinterpret_cast<const u32x4_t*>(ws.T + (item0 + c) * kGdrPieceHalves);
    const u32x4_t* Pm = reinterpret_cast<const u32x4_t*>(ws.Pm + (item0 + c) * kGdrPieceHalves);
#pragma unroll
    for (int i = 0; i < W::NTL; ++i) {
      const int e = i * NT + tid;
      if (W::kT / 8 % NT == 0 || e < W::kT / 8) tr[i] = T[e];
    }
#pragma unroll
    for (int i = 0; i < W::NPL; ++i) {
      const int e = i * NT + tid;
      // with one half a piece, every other 64 of the workspace's
      const int from = OP == 2 ? e : 2 * e - (e & 63);
      if (W::kP / 8 % NT == 0 || e < W::kP / 8) pr[i] = Pm[from];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * NT + tid;
      if (5 * kGdrC % NT == 0 || e < 5 * kGdrC) fr[i] = fac[kFacK * kGdrC + e];
    }
    fend = fac[kFacEnd * kGdrC];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t off = (static_cast<uint32_t>(16 * tt + 4 * g + i) * vs + static_cast<uint32_t>(col)) * EB;
        vr[4 * tt + i] = buffer_load_bits<BF16>(rv, col_ok ? off : kOutOfRange);
      }
    }
  };
  auto stage = [&](int buf) __attribute__((always_inline)) {
    _Float16* sK = reinterpret_cast<_Float16*>(lds[buf]);
    _Float16* sQ = sK + W::kMat;
    u32x4_t* sT = reinterpret_cast<u32x4_t*>(KEEP ? sQ : sQ + W::kMat);
    u32x4_t* sP = sT + W::kT / 8;
    float* sF = reinterpret_cast<float*>(sP + W::kP / 8);
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
      if constexpr (KEEP) continue;
      raw8_values<BF16, VEC>(qr[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= qu[i];
      hi = halves(x);
      *reinterpret_cast<half8_t*>(sQ + t * RS + n) = hi;
      if constexpr (RAW == 2) *reinterpret_cast<half8_t*>(sQ + kGdrC * RS + t * RS + n) = rest(x, hi);
    }
#pragma unroll
    for (int i = 0; i < W::NTL; ++i) {
      const int e = i * NT + tid;
      if (W::kT / 8 % NT == 0 || e < W::kT / 8) sT[e] = tr[i];
    }
#pragma unroll
    for (int i = 0; i < W::NPL; ++i) {
      const int e = i * NT + tid;
      if (W::kP / 8 % NT == 0 || e < W::kP / 8) sP[e] = pr[i];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * NT + tid;
      if (5 * kGdrC % NT == 0 || e < 5 * kGdrC) sF[e] = fr[i];
    }
    if (tid == 0) sF[5 * kGdrC] = fend;
  };

  if (n_chunks > 0) {
    fetch(0);
    stage(0);
  }
  __syncthreads();
  half8_t Sh[NK], Sl[NK];
  Pow2 ss = pow2_to_top(tiles_absmax<NJ>(S));
#pragma unroll
  for (int q = 0; q < NK; ++q) tiles_to_operand<true>(S[2 * q], S[2 * q + 1], ss.up, Sh[q], Sl[q]);

  for (int c = 0; c < n_chunks; ++c) {
    const int buf = W::NBUF == 2 ? (c & 1) : 0;
    const _Float16* sK = reinterpret_cast<const _Float16*>(lds[buf]);
    const _Float16* sQ = sK + W::kMat;
    const _Float16* sT = KEEP ? sQ : sQ + W::kMat;
    const _Float16* sP = sT + W::kT;
    const float* sF = reinterpret_cast<const float*>(sP + W::kP);
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = bits_to_f32<BF16>(vr[i]);
    if (c + 1 < n_chunks) fetch(c + 1);
    if constexpr (KEEP) {
      const int64_t item = item0 + c;
      if (col_ok) {
        float* dst = ws.S + (item * P + col) * N;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int n = 32 * (j / 2) + 8 * g + 4 * (j & 1);
          if (N % 4 == 0) {
            if (n < N) *reinterpret_cast<f32x4_t*>(dst + n) = S[j];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (n + i < N) dst[n + i] = S[j][i];
            }
          }
        }
      }
      const float top = lanes16_max(tiles_absmax<NJ>(S));
      if (lane == 0 && col < P) ws.top[(item * kGdrMaxima + kMaxS) * kGdrMaxSlices + col / 16] = top;
    }

    // K S and Q S
    f32x4_t ks[4], qs[4];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) ks[tt] = qs[tt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < NK; ++q) {
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int at = (16 * tt + m) * RS + 32 * q + 8 * g;
        const half8_t a = *reinterpret_cast<const half8_t*>(sK + at);
        ks[tt] = mfma16(a, Sh[q], ks[tt]);
        ks[tt] = mfma16(a, Sl[q], ks[tt]);
        if constexpr (RAW == 2) {
          ks[tt] = mfma16(*reinterpret_cast<const half8_t*>(sK + kGdrC * RS + at), Sh[q], ks[tt]);
        }
        if constexpr (KEEP) continue;
        const half8_t aq = *reinterpret_cast<const half8_t*>(sQ + at);
        qs[tt] = mfma16(aq, Sh[q], qs[tt]);
        if constexpr (OP == 2) {
          qs[tt] = mfma16(aq, Sl[q], qs[tt]);
          if constexpr (RAW == 2) {
            qs[tt] = mfma16(*reinterpret_cast<const half8_t*>(sQ + kGdrC * RS + at), Sh[q], qs[tt]);
          }
        }
      }
    }
    // R = V - diag(e^c) K S, then E = T R
    f32x4_t R[4];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      const f32x4_t f = *reinterpret_cast<const f32x4_t*>(sF + 0 * kGdrC + 16 * tt + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) R[tt][i] = fmaf(-(f[i] * ss.down), ks[tt][i], v[4 * tt + i]);
    }
    f32x4_t E[4];
    {
      const Pow2 sr = pow2_to_top(tiles_absmax<4>(R));
      half8_t Rh[2], Rl[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) tiles_to_operand<true>(R[2 * q], R[2 * q + 1], sr.up, Rh[q], Rl[q]);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        E[tt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q <= tt / 2; ++q) {
          const _Float16* at = sT + gdr_frag(tt, q) * 2 * kGdrFragHalves + lane * 8;
          const half8_t hi = *reinterpret_cast<const half8_t*>(at);
          const half8_t lo = *reinterpret_cast<const half8_t*>(at + kGdrFragHalves);
          E[tt] = mfma16(hi, Rh[q], E[tt]);
          E[tt] = mfma16(hi, Rl[q], E[tt]);
          E[tt] = mfma16(lo, Rh[q], E[tt]);
        }
        const f32x4_t f = *reinterpret_cast<const f32x4_t*>(sF + 3 * kGdrC + 16 * tt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) E[tt][i] *= f[i] * sr.down;
      }
    }
    // S' = e^(c_end) S + K^T (w E)
    {
      f32x4_t D[4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const f32x4_t f = *reinterpret_cast<const f32x4_t*>(sF + 2 * kGdrC + 16 * tt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) D[tt][i] = E[tt][i] * f[i];
      }
      const Pow2 sd = pow2_to_top(tiles_absmax<4>(D));
      half8_t Dh[2], Dl[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) tiles_to_operand<true>(D[2 * q], D[2 * q + 1], sd.up, Dh[q], Dl[q]);
      const float end = sF[5 * kGdrC];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          // rows 32 q + 4 g + m / 4 (and + 16), columns of tile j in its order
          const int at = (32 * q + 4 * g + (m >> 2)) * RS + 32 * (j / 2) + 8 * (m & 3) + 4 * (j & 1);
          const half4_t a0 = lds_column4(sK + at), a1 = lds_column4(sK + at + 16 * RS);
          const half8_t a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
          acc = mfma16(a, Dh[q], acc);
          acc = mfma16(a, Dl[q], acc);
          if constexpr (RAW == 2) {
            const half4_t b0 = lds_column4(sK + kGdrC * RS + at), b1 = lds_column4(sK + kGdrC * RS + at + 16 * RS);
            acc = mfma16(__builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7), Dh[q], acc);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) S[j][i] = fmaf(acc[i], sd.down, end * S[j][i]);
      }
    }
    if constexpr (KEEP) {
      const int64_t item = item0 + c;
      float* dst = ws.E + item * kGdrC * P;
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (col_ok) dst[(16 * tt + 4 * g + i) * P + col] = E[tt][i];
        }
      }
      const float top = lanes16_max(tiles_absmax<4>(E));
      if (lane == 0 && col < P) ws.top[(item * kGdrMaxima + kMaxE) * kGdrMaxSlices + col / 16] = top;
    }
    // Y = diag(scale e^c) Q S + Pm E (S: the state before)
    if constexpr (!KEEP) {
      const Pow2 se = pow2_to_top(tiles_absmax<4>(E));
      half8_t Eh[2], El[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) tiles_to_operand<OP == 2>(E[2 * q], E[2 * q + 1], se.up, Eh[q], El[q]);
      const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
      const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
      const int out_rows = static_cast<int>(L - t0 < kGdrC ? L - t0 : kGdrC);
      const rsrc_t ry = rows_buffer<OB16 ? 2 : 4>(p.y, (row_b + t0) * yrow + static_cast<int64_t>(h) * P, out_rows,
                                                  yrow, P);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q <= tt / 2; ++q) {
          const _Float16* at = sP + gdr_frag(tt, q) * OP * kGdrFragHalves + lane * 8;
          const half8_t hi = *reinterpret_cast<const half8_t*>(at);
          acc = mfma16(hi, Eh[q], acc);
          if constexpr (OP == 2) {
            acc = mfma16(hi, El[q], acc);
            acc = mfma16(*reinterpret_cast<const half8_t*>(at + kGdrFragHalves), Eh[q], acc);
          }
        }
        const f32x4_t fq = *reinterpret_cast<const f32x4_t*>(sF + 1 * kGdrC + 16 * tt + 4 * g);
        const f32x4_t fp = *reinterpret_cast<const f32x4_t*>(sF + 4 * kGdrC + 16 * tt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * tt + 4 * g + i;
          const float y = fmaf(fq[i] * ss.down, qs[tt][i], fp[i] * se.down * acc[i]);
          const uint32_t off = (static_cast<uint32_t>(t) * yrow + static_cast<uint32_t>(col)) * (OB16 ? 2 : 4);
          buffer_store_f32<OB16>(t < rows ? y : 0.0f, ry, col_ok ? off : kOutOfRange);
        }
      }
    }
    ss = pow2_to_top(tiles_absmax<NJ>(S));
#pragma unroll
    for (int q = 0; q < NK; ++q) tiles_to_operand<true>(S[2 * q], S[2 * q + 1], ss.up, Sh[q], Sl[q]);

    if constexpr (W::NBUF == 1) __syncthreads();
    if (c + 1 < n_chunks) stage(W::NBUF == 2 ? ((c + 1) & 1) : 0);
    __syncthreads();
  }

  if constexpr (KEEP) return;
  // Steps behind the row's last: zeros from the first chunk that was not walked.
  for (int64_t t = static_cast<int64_t>(n_chunks) * kGdrC + g; t < L; t += 4) {
    if (col_ok) store_elem<OB16>(p.y, (row_b + t) * yrow + static_cast<int64_t>(h) * P + col, 0.0f);
  }
  if (p.h_final != nullptr && col_ok) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
        if (n < N) p.h_final[sb + n] = S[j][i];
      }
    }
  }
}

template <int NP, bool BF16, bool OB16, bool VEC, bool KEEP>
void gdr_launch_chunk_nw(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, hipStream_t st) {
  const int64_t bh = a.batch * a.nheads;
  const int64_t slices = (a.headdim + 15) / 16;
  if (slices <= 2) {
    gdr_chunk_kernel<NP, BF16, OB16, VEC, 2, KEEP>
        <<<static_cast<unsigned>(bh * ((slices + 1) / 2)), 128, 0, st>>>(a, ws, chunks);
  } else {
    gdr_chunk_kernel<NP, BF16, OB16, VEC, 4, KEEP>
        <<<static_cast<unsigned>(bh * ((slices + 3) / 4)), 256, 0, st>>>(a, ws, chunks);
  }
}

template <bool BF16>
int gdr_launch_chunk(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, bool backward, bool vec, hipStream_t st) {
  const auto types = [&](auto np) {
    constexpr int NP = decltype(np)::value;
    if (backward) {
      vec ? gdr_launch_chunk_nw<NP, BF16, true, true, true>(a, ws, chunks, st)
          : gdr_launch_chunk_nw<NP, BF16, true, false, true>(a, ws, chunks, st);
    } else if (a.out_bf16) {
      vec ? gdr_launch_chunk_nw<NP, BF16, true, true, false>(a, ws, chunks, st)
          : gdr_launch_chunk_nw<NP, BF16, true, false, false>(a, ws, chunks, st);
    } else {
      vec ? gdr_launch_chunk_nw<NP, BF16, false, true, false>(a, ws, chunks, st)
          : gdr_launch_chunk_nw<NP, BF16, false, false, false>(a, ws, chunks, st);
    }
  };
  if (a.dstate <= 64) {
    types(std::integral_constant<int, 64>{});
  } else {
    types(std::integral_constant<int, 128>{});
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
