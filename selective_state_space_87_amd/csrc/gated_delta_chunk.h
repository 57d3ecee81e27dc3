// Gated delta rule, the walk over a head's chunks (see gdr_mma.h for the
// chunk's equations, operand halves and layouts). Included by one source file
// per input type.
//
// Sixteen columns of a head's state [N, P] belong to a pair of waves for the
// whole sequence. A chunk is a chain of products on them,
//   K S, Q S  ->  E = T (V - ..)  ->  Y = .. + Pm E,  S' = .. + K^T (w E)
// and the pair splits every link: of the products with K, Q, T and Pm wave r of
// the pair takes the 32 steps 32 r .. + 31, of the state's update the half
// r of the N rows. What one needs of the other goes through LDS as the operand
// halves it is used as (S, and R and E of the first 32 steps, and w E), three
// barriers a chunk. A chain as long as this is bound by what one wave can
// issue, not by the units: with one wave a slice a chunk of the layer
// (4, 8192, 32 heads of 128 x 128) took 13 000 clocks, of which the vector ALU
// worked 4 100 and the matrix unit 1 660.
//
// A block of NPAIR pairs (16 NPAIR columns) shares the halves of K and Q and
// the factors through LDS; the next chunk's are in flight in
// registers meanwhile, and go into the other LDS buffer where two fit. T and
// Pm are read by a wave straight into the registers it feeds them from.
#pragma once

#include "gdr_mma.h"

namespace ssm {

// KEEP: the backward's pass over the chunks, which leaves the entering states
// and E in the workspace and no y (neither Q nor Pm is touched).
template <int NP, bool BF16, bool OB16, int NPAIR, bool KEEP>
struct GdrWalk {
  static constexpr int NT = 128 * NPAIR;
  static constexpr int RAW = BF16 ? 1 : 2;
  static constexpr int OP = OB16 ? 1 : 2;               // halves in the products that only y sees
  static constexpr int kMat = RAW * kGdrC * NP;         // halves of K (or Q)
  static constexpr int kFac = 4 * kGdrC + 4;            // K, Q, W, P factors and the end's
  static constexpr int kBufBytes = (KEEP ? 1 : 2) * kMat * 2 + kFac * 4;
  // a pair's exchange, in halves: S (NP / 32 pieces), R, w E (2), E; then scales (floats, a lane each)
  static constexpr int kXS = 0, kXR = kXS + NP / 32 * 2 * kGdrFragHalves, kXD = kXR + 2 * kGdrFragHalves;
  static constexpr int kXE = kXD + 4 * kGdrFragHalves, kXF = kXE + OP * kGdrFragHalves;
  static constexpr int kPairBytes = kXF * 2 + 6 * 64 * 4;
  static constexpr int NBUF = 2 * kBufBytes + NPAIR * kPairBytes <= 160 * 1024 ? 2 : 1;
  static constexpr int NKQ = kMat / 8 / NT;             // 16-byte pieces of K (and Q) a thread
  static constexpr int NFL = (4 * kGdrC + NT - 1) / NT;
};

template <int NP, bool BF16, bool OB16, int NPAIR, bool KEEP>
__global__ __launch_bounds__(128 * NPAIR, NPAIR == 4 ? 2 : 1) void gdr_chunk_kernel(const GatedDeltaArgs p,
                                                                                    const GdrWork ws, int chunks) {
  using W = GdrWalk<NP, BF16, OB16, NPAIR, KEEP>;
  constexpr int NT = W::NT, RAW = W::RAW, OP = W::OP;
  constexpr int kLo = kGdrC * NP;                       // from an element's hi half to its lo half
  constexpr int NJ = NP / 32, NK = NP / 64;             // state tiles and operand pieces of a wave
  constexpr int EB = BF16 ? 2 : 4;
  __shared__ __align__(16) char lds[W::NBUF][W::kBufBytes];
  __shared__ __align__(16) char xch[NPAIR][W::kPairBytes];

  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pr = w >> 1, r = w & 1;
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads);
  const int N = static_cast<int>(p.dstate), P = static_cast<int>(p.headdim);
  const int pblocks = (P + 16 * NPAIR - 1) / (16 * NPAIR);
  const int bh = static_cast<int>(blockIdx.x) / pblocks;
  const int b = bh / H, h = bh % H, kh = h / (H / G);
  const int col = (static_cast<int>(blockIdx.x) % pblocks) * 16 * NPAIR + 16 * pr + m;
  const bool col_ok = col < P;
  const int64_t L = p.seqlen;
  const int64_t len = gdr_row_steps(p.seqlens, b, L);
  const int n_chunks = static_cast<int>((len + kGdrC - 1) / kGdrC);
  const int64_t row_b = static_cast<int64_t>(b) * L;
  const int64_t item0 = static_cast<int64_t>(bh) * chunks, kv0 = (static_cast<int64_t>(b) * G + kh) * chunks;
  const int64_t sb = (static_cast<int64_t>(bh) * P + (col_ok ? col : 0)) * N;
  const uint32_t yrow = static_cast<uint32_t>(H * P);

  _Float16* const xh = reinterpret_cast<_Float16*>(xch[pr]);
  float* const xf = reinterpret_cast<float*>(xh + W::kXF);
  float *const xs_f = xf, *const xr_f = xf + 128, *const xd_f = xf + 192, *const xe_f = xf + 320;
  const auto piece = [&](int at, int q, int half, int halves_a_piece) __attribute__((always_inline)) {
    return reinterpret_cast<half8_t*>(xh + at + (q * halves_a_piece + half) * kGdrFragHalves + lane * 8);
  };

  // The state: tile j = 2 q + u of the wave's half, element i is n = n0 + 32 q
  // + 8 g + 4 u + i of column `col`, so that tiles 2 q and 2 q + 1 together are
  // n = 32 q + 8 g + 0..7: the contraction order in which a lane's piece of a K
  // row is contiguous.
  const int n0 = r * (NP / 2);
  f32x4_t S[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
      S[j][i] = (p.h0 != nullptr && col_ok && n < N) ? p.h0[sb + n] : 0.0f;
    }
  }

  u32x4_t kr[W::NKQ], qr[W::NKQ];
  float fr[W::NFL];
  float fend = 0.0f, ftri = 0.0f, fend_next = 0.0f, ftri_next = 0.0f;
  half8_t Td[2][2], To[2][2], Pd[2][OP], Po[2][OP];  // pieces on the diagonal, and left of it (wave 1)
  uint32_t vr[8];

  // Rows of K and Q, factors and the wave's rows of V.
  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
    const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
    const int64_t row0 = row_b + t0;
    const uint32_t vs = static_cast<uint32_t>(p.v_step);
    const rsrc_t rv = rows_buffer<EB>(p.v, row0 * p.v_step + static_cast<int64_t>(h) * P, rows, vs, P);
    const float* fac = ws.fac + (item0 + c) * (kGdrFactors * kGdrC);
    const u32x4_t* K = reinterpret_cast<const u32x4_t*>(ws.K + (kv0 + c) * W::kMat) + tid;
    const u32x4_t* Q = reinterpret_cast<const u32x4_t*>(ws.Q + (kv0 + c) * W::kMat) + tid;
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      kr[i] = K[i * NT];
      if constexpr (!KEEP) qr[i] = Q[i * NT];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * NT + tid;
      fr[i] = fac[kFacK * kGdrC + (4 * kGdrC % NT == 0 ? e : e % (4 * kGdrC))];
    }
    fend_next = fac[kFacEnd * kGdrC];
    ftri_next = fac[kFacEnd * kGdrC + 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = 32 * r + 16 * (i / 4) + 4 * g + (i % 4);
      const uint32_t off = (static_cast<uint32_t>(t) * vs + static_cast<uint32_t>(col)) * EB;
      vr[i] = buffer_load_bits<BF16>(rv, col_ok ? off : kOutOfRange);
    }
  };
  // The wave's pieces of T: row tiles 2 r and 2 r + 1.
  auto fetch_T = [&](int c) __attribute__((always_inline)) {
    const half8_t* src = reinterpret_cast<const half8_t*>(ws.T + (item0 + c) * kGdrPieceHalves) + lane;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int f = r == 0 ? u : 3 + 2 * u;
      Td[u][0] = src[(2 * f) * 64];
      Td[u][1] = src[(2 * f + 1) * 64];
      const int o = r == 0 ? f : 2 + 2 * u;  // (wave 0 has none: any of its own)
      To[u][0] = src[(2 * o) * 64];
      To[u][1] = src[(2 * o + 1) * 64];
    }
  };
  auto fetch_P = [&](int c) __attribute__((always_inline)) {
    if constexpr (KEEP) return;
    const half8_t* src = reinterpret_cast<const half8_t*>(ws.Pm + (item0 + c) * kGdrPieceHalves) + lane;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int f = r == 0 ? u : 3 + 2 * u;
      Pd[u][0] = src[(2 * f) * 64];
      if constexpr (OP == 2) Pd[u][OP - 1] = src[(2 * f + 1) * 64];
      const int o = r == 0 ? f : 2 + 2 * u;
      Po[u][0] = src[(2 * o) * 64];
      if constexpr (OP == 2) Po[u][OP - 1] = src[(2 * o + 1) * 64];
    }
  };
  auto stage = [&](int buf) __attribute__((always_inline)) {
    _Float16* sK = reinterpret_cast<_Float16*>(lds[buf]);
    _Float16* sQ = sK + W::kMat;
    float* sF = reinterpret_cast<float*>(KEEP ? sQ : sQ + W::kMat);
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      reinterpret_cast<u32x4_t*>(sK)[i * NT + tid] = kr[i];
      if constexpr (!KEEP) reinterpret_cast<u32x4_t*>(sQ)[i * NT + tid] = qr[i];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * NT + tid;
      if (4 * kGdrC % NT == 0 || e < 4 * kGdrC) sF[e] = fr[i];
    }
    fend = fend_next;
    ftri = ftri_next;
  };

  half8_t Sh[NK], Sl[NK];
  float s_down = 0.0f;
  // The wave's half of S as an operand, for itself and for the other.
  auto split_S = [&]() __attribute__((always_inline)) {
    const Pow2 s = pow2_to_top(tiles_absmax<NJ>(S));
    s_down = s.down;
#pragma unroll
    for (int q = 0; q < NK; ++q) {
      tiles_to_operand<true>(S[2 * q], S[2 * q + 1], s.up, Sh[q], Sl[q]);
      *piece(W::kXS, r * NK + q, 0, 2) = Sh[q];
      *piece(W::kXS, r * NK + q, 1, 2) = Sl[q];
    }
    xs_f[64 * r + lane] = s.down;
  };

  if (n_chunks > 0) {
    fetch(0);
    fetch_T(0);
    fetch_P(0);
    stage(0);
  }
  split_S();
  __syncthreads();

  for (int c = 0; c < n_chunks; ++c) {
    const int buf = W::NBUF == 2 ? (c & 1) : 0;
    const _Float16* sK = reinterpret_cast<const _Float16*>(lds[buf]);
    const _Float16* sQ = sK + W::kMat;
    const float* sF = reinterpret_cast<const float*>(KEEP ? sQ : sQ + W::kMat);
    const auto factor = [&](int which, int u) __attribute__((always_inline)) {
      return *reinterpret_cast<const f32x4_t*>(sF + which * kGdrC + 32 * r + 16 * u + 4 * g);
    };
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bits_to_f32<BF16>(vr[i]);
    // The loads of the next chunk stand in no branch (behind the last chunk they
    // fetch it again): a conditional load is waited for where the branches join.
    const bool more = c + 1 < n_chunks;
    const int next = more ? c + 1 : c;
    fetch(next);
    if constexpr (KEEP) {
      const int64_t item = item0 + c;
      if (col_ok) {
        float* dst = ws.S + (item * P + col) * N;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1);
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
      if (lane == 0 && col < P) ws.top[(item * kGdrMaxima + kMaxS) * kGdrMaxSlots + col / 16 * 2 + r] = top;
    }

    // K S and Q S on the wave's 32 steps: its own half of S, and the other's.
    f32x4_t ks[2][2], qs[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int o = 0; o < 2; ++o) ks[o][u] = qs[o][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
#pragma unroll
      for (int q = 0; q < NK; ++q) {
        const int f = (o == 0 ? r : 1 - r) * NK + q;
        const half8_t sh = o == 0 ? Sh[q] : *piece(W::kXS, f, 0, 2);
        const half8_t sl = o == 0 ? Sl[q] : *piece(W::kXS, f, 1, 2);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int at = kq_at<NP>(32 * r + 16 * u + m, 32 * f + 8 * g);
          const half8_t a = *reinterpret_cast<const half8_t*>(sK + at);
          ks[o][u] = mfma16(a, sh, ks[o][u]);
          ks[o][u] = mfma16(a, sl, ks[o][u]);
          if constexpr (RAW == 2) {
            ks[o][u] = mfma16(*reinterpret_cast<const half8_t*>(sK + kLo + at), sh, ks[o][u]);
          }
          if constexpr (KEEP) continue;
          const half8_t aq = *reinterpret_cast<const half8_t*>(sQ + at);
          qs[o][u] = mfma16(aq, sh, qs[o][u]);
          if constexpr (OP == 2) {
            qs[o][u] = mfma16(aq, sl, qs[o][u]);
            if constexpr (RAW == 2) {
              qs[o][u] = mfma16(*reinterpret_cast<const half8_t*>(sQ + kLo + at), sh, qs[o][u]);
            }
          }
        }
      }
    }
    const float so_down = xs_f[64 * (1 - r) + lane], ss_down = s_down;
    // R = V - diag(e^c) K S; the first 32 steps' also for the other wave.
    half8_t Rh, Rl;
    Pow2 sr;
    {
      f32x4_t R[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4_t f = factor(0, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          R[u][i] = fmaf(-f[i], fmaf(ks[1][u][i], so_down, ks[0][u][i] * ss_down), v[4 * u + i]);
        }
      }
      sr = pow2_to_top(tiles_absmax<2>(R));
      tiles_to_operand<true>(R[0], R[1], sr.up, Rh, Rl);
      if (r == 0) {
        *piece(W::kXR, 0, 0, 2) = Rh;
        *piece(W::kXR, 0, 1, 2) = Rl;
        xr_f[lane] = sr.down;
      }
    }
    __syncthreads();

    // E = T R
    f32x4_t E[2];
    {
      const float down = sr.down * ftri;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        acc = mfma16(Td[u][0], Rh, acc);
        acc = mfma16(Td[u][0], Rl, acc);
        acc = mfma16(Td[u][1], Rh, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) E[u][i] = acc[i] * down;
      }
      if (r == 1) {
        const half8_t oh = *piece(W::kXR, 0, 0, 2), ol = *piece(W::kXR, 0, 1, 2);
        const float other = xr_f[lane] * ftri;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          acc = mfma16(To[u][0], oh, acc);
          acc = mfma16(To[u][0], ol, acc);
          acc = mfma16(To[u][1], oh, acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) E[u][i] = fmaf(acc[i], other, E[u][i]);
        }
      }
    }
    fetch_T(next);
    // w E as an operand for both waves, E for the wave of the later steps.
    half8_t Dh, Dl, Eh, El;
    Pow2 sd, se;
    {
      f32x4_t D[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4_t f = factor(2, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) D[u][i] = E[u][i] * f[i];
      }
      sd = pow2_to_top(tiles_absmax<2>(D));
      tiles_to_operand<true>(D[0], D[1], sd.up, Dh, Dl);
      *piece(W::kXD, r, 0, 2) = Dh;
      *piece(W::kXD, r, 1, 2) = Dl;
      xd_f[64 * r + lane] = sd.down;
      if constexpr (KEEP) {
        const int64_t item = item0 + c;
        float* dst = ws.E + item * kGdrC * P;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (col_ok) dst[(32 * r + 16 * (i / 4) + 4 * g + (i % 4)) * P + col] = E[i / 4][i % 4];
        }
        const float top = lanes16_max(tiles_absmax<2>(E));
        if (lane == 0 && col < P) ws.top[(item * kGdrMaxima + kMaxE) * kGdrMaxSlots + col / 16 * 2 + r] = top;
      } else {
        se = pow2_to_top(tiles_absmax<2>(E));
        tiles_to_operand<OP == 2>(E[0], E[1], se.up, Eh, El);
        if (r == 0) {
          *piece(W::kXE, 0, 0, OP) = Eh;
          if constexpr (OP == 2) *piece(W::kXE, 0, OP - 1, OP) = El;
          xe_f[lane] = se.down;
        }
      }
    }
    __syncthreads();

    // S' = e^(c_end) S + K^T (w E) on the wave's half of the rows
    {
      const half8_t oh = *piece(W::kXD, 1 - r, 0, 2), ol = *piece(W::kXD, 1 - r, 1, 2);
      const float d_own = sd.down, d_oth = xd_f[64 * (1 - r) + lane];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        f32x4_t acc[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          acc[o] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          const half8_t dh = o == 0 ? Dh : oh, dl = o == 0 ? Dl : ol;
          // rows 32 q + 4 g + m / 4 (and + 16), columns of tile j in its order
          const int at = kq_at<NP>(32 * (o == 0 ? r : 1 - r) + 4 * g + (m >> 2), n0 + 32 * (j / 2) + 8 * (m & 3)) + 4 * (j & 1);
          const half4_t a0 = lds_column4(sK + at), a1 = lds_column4(sK + at + 16 * NP);
          const half8_t a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
          acc[o] = mfma16(a, dh, acc[o]);
          acc[o] = mfma16(a, dl, acc[o]);
          if constexpr (RAW == 2) {
            const half4_t b0 = lds_column4(sK + kLo + at), b1 = lds_column4(sK + kLo + at + 16 * NP);
            acc[o] = mfma16(__builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7), dh, acc[o]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) S[j][i] = fmaf(acc[1][i], d_oth, fmaf(acc[0][i], d_own, fend * S[j][i]));
      }
    }
    // Y = diag(scale e^c) Q S + Pm E (S: the state before)
    if constexpr (!KEEP) {
      const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
      const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
      const int out_rows = static_cast<int>(L - t0 < kGdrC ? L - t0 : kGdrC);
      const rsrc_t ry = rows_buffer<OB16 ? 2 : 4>(p.y, (row_b + t0) * yrow + static_cast<int64_t>(h) * P, out_rows,
                                                  yrow, P);
      f32x4_t pe[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        acc = mfma16(Pd[u][0], Eh, acc);
        if constexpr (OP == 2) {
          acc = mfma16(Pd[u][0], El, acc);
          acc = mfma16(Pd[u][OP - 1], Eh, acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) pe[u][i] = acc[i] * se.down;
      }
      if (r == 1) {
        const half8_t oh = *piece(W::kXE, 0, 0, OP);
        const float other = xe_f[lane];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          acc = mfma16(Po[u][0], oh, acc);
          if constexpr (OP == 2) {
            acc = mfma16(Po[u][0], *piece(W::kXE, 0, OP - 1, OP), acc);
            acc = mfma16(Po[u][OP - 1], oh, acc);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) pe[u][i] = fmaf(acc[i], other, pe[u][i]);
        }
      }
      fetch_P(next);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4_t fq = factor(1, u), fp = factor(3, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 32 * r + 16 * u + 4 * g + i;
          const float y = fmaf(fq[i], fmaf(qs[1][u][i], so_down, qs[0][u][i] * ss_down), fp[i] * pe[u][i]);
          const uint32_t off = (static_cast<uint32_t>(t) * yrow + static_cast<uint32_t>(col)) * (OB16 ? 2 : 4);
          buffer_store_f32<OB16>(t < rows ? y : 0.0f, ry, col_ok ? off : kOutOfRange);
        }
      }
    }
    if (more) split_S();
    if constexpr (W::NBUF == 1) __syncthreads();
    if (more) stage(W::NBUF == 2 ? ((c + 1) & 1) : 0);
    __syncthreads();
  }

  if constexpr (KEEP) return;
  // Steps behind the row's last: zeros from the first chunk that was not walked.
  for (int64_t t = static_cast<int64_t>(n_chunks) * kGdrC + 4 * r + g; t < L; t += 8) {
    if (col_ok) store_elem<OB16>(p.y, (row_b + t) * yrow + static_cast<int64_t>(h) * P + col, 0.0f);
  }
  if (p.h_final != nullptr && col_ok) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
        if (n < N) p.h_final[sb + n] = S[j][i];
      }
    }
  }
}

template <int NP, bool BF16, bool OB16, bool KEEP>
void gdr_launch_chunk_pairs(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, hipStream_t st) {
  const int64_t bh = a.batch * a.nheads;
  const int64_t slices = (a.headdim + 15) / 16;
  const int pairs = gdr_block_pairs(bh, slices);
  const auto blocks = [&](int n) { return static_cast<unsigned>(bh * ((slices + n - 1) / n)); };
  if (pairs == 1) {
    gdr_chunk_kernel<NP, BF16, OB16, 1, KEEP><<<blocks(1), 128, 0, st>>>(a, ws, chunks);
  } else if (pairs == 2) {
    gdr_chunk_kernel<NP, BF16, OB16, 2, KEEP><<<blocks(2), 256, 0, st>>>(a, ws, chunks);
  } else {
    gdr_chunk_kernel<NP, BF16, OB16, 4, KEEP><<<blocks(4), 512, 0, st>>>(a, ws, chunks);
  }
}

template <bool BF16>
int gdr_launch_chunk(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, bool backward, hipStream_t st) {
  const auto types = [&](auto np) {
    constexpr int NP = decltype(np)::value;
    if (backward) {
      gdr_launch_chunk_pairs<NP, BF16, true, true>(a, ws, chunks, st);
    } else if (a.out_bf16) {
      gdr_launch_chunk_pairs<NP, BF16, true, false>(a, ws, chunks, st);
    } else {
      gdr_launch_chunk_pairs<NP, BF16, false, false>(a, ws, chunks, st);
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
