// Gated delta rule backward, the walk back over a head's chunks (see gdr_mma.h).
// With the gradient X of the state leaving a chunk, dY the output's:
//   U  = Pm^T dY + diag(w) K X            (of E, as the later ones see it)
//   dE = T^T U                            (of V - diag(e^c) K S; also dV)
//   X' = e^(c_end) X + Q^T (qf dY) - K^T (kf dE)
// the mirror image of the forward's walk, and split the same way: a pair of
// waves owns 16 columns of X in registers; wave r takes steps 32 r .. + 31 of
// K X and of the second line, and half r of the N rows of the third. Through
// LDS go X (both ways), U of the last 32 steps (to the wave of the first) and
// kf dE (both ways). What does not depend on X is made by two more waves a
// pair, a chunk ahead: Pm^T dY and Q^T (qf dY), which the state's waves add from
// LDS, and all loads (when it was built, alone, 202 us for (2, 4096, 16 heads of
// 128 x 128), 253 with a pair's own waves doing it). X is left in the workspace for every chunk (the gradient
// of its leaving state), dE in dv. Every other slice is walked with the other sign
// (see gdr_mma.h), and its X is left so.
#include <hip/hip_runtime.h>

#include "gated_delta_chunk.h"
#include "gdr_mma.h"

namespace ssm {

namespace {

template <int NP, bool BF16, int NPAIR>
struct GdrBack {
  static constexpr int NT = 256 * NPAIR;
  static constexpr int NL = 128 * NPAIR;                // threads that load
  static constexpr int RAW = BF16 ? 1 : 2;
  static constexpr int kMat = RAW * kGdrC * NP;
  static constexpr int kTri = kGdrPieceHalves;
  static constexpr int kFac = 4 * kGdrC + 4;            // K, Q, W, P factors; the end's and T's
  static constexpr int kBufBytes = kMat * 2;            // K (Q is read in a chunk's first phase alone: one buffer)
  // a pair's exchange, in halves: X (NP / 32 pieces), U, kf dE of either wave;
  // then floats: Pm^T dY (4 tiles), Q^T (qf dY) (NP / 16 tiles), scales
  static constexpr int kXX = 0, kXU = kXX + NP / 32 * 2 * kGdrFragHalves, kXB = kXU + 2 * kGdrFragHalves;
  static constexpr int kXH = kXB + 4 * kGdrFragHalves;
  static constexpr int kFY = 0, kFQ = kFY + 4 * 256, kFS = kFQ + NP / 16 * 256;
  static constexpr int kPairBytes = kXH * 2 + (kFS + 5 * 64) * 4;
  static constexpr int kFixed = kMat * 2 + kTri * 2 + 2 * kFac * 4 + NPAIR * kPairBytes;
  static constexpr int NBUF = 2 * kBufBytes + kFixed <= 160 * 1024 ? 2 : 1;
  static constexpr int NKQ = kMat / 8 / NL;
  static constexpr int NTL = kTri / 8 / NL;
  static constexpr int NFL = (4 * kGdrC + NL - 1) / NL;
};

template <class W, int NPAIR>
struct GdrBackLds {
  __align__(16) char k[W::NBUF][W::kBufBytes];
  __align__(16) _Float16 Q[W::kMat];
  __align__(16) _Float16 T[W::kTri];
  __align__(16) float fac[2][W::kFac];
  __align__(16) char xch[NPAIR][W::kPairBytes];
};

// The walk of block `block`, by threads 0 .. W::NT - 1 (tid). Its barriers: two,
// and three a chunk (four with one buffer).
template <int NP, bool BF16, int NPAIR>
__device__ __forceinline__ void gdr_walk_back(const GatedDeltaBwdArgs& a, const GdrWork& ws, int chunks, int block, int tid,
                                              GdrBackLds<GdrBack<NP, BF16, NPAIR>, NPAIR>& sh) {
  using W = GdrBack<NP, BF16, NPAIR>;
  constexpr int RAW = W::RAW, NJ = NP / 32, NK = NP / 64;
  constexpr int kLo = kGdrC * NP;
  auto& lds = sh.k;
  auto& sFac = sh.fac;
  auto& xch = sh.xch;
  _Float16 *const sQ = sh.Q, *const sT = sh.T;
  const GatedDeltaArgs& p = a.f;

  const int lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pr = (w >> 1) % NPAIR, r = w & 1;
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads);
  const int N = static_cast<int>(p.dstate), P = static_cast<int>(p.headdim);
  const int pblocks = (P + 16 * NPAIR - 1) / (16 * NPAIR);
  const int place = gdr_xcd_place(block, static_cast<int>(gridDim.x), H / G * pblocks);
  const int bh = place / pblocks;
  const int b = bh / H, h = bh % H, kh = h / (H / G);
  const int col = (place % pblocks) * 16 * NPAIR + 16 * pr + m;
  const bool col_ok = col < P;
  const int odd = (col >> 4) & 1;  // the slice's X, dY and U are taken negative, and X is left so
  const int64_t L = p.seqlen;
  const int64_t len = gdr_row_steps(p.seqlens, b, L);
  const int n_chunks = static_cast<int>((len + kGdrC - 1) / kGdrC);
  const int64_t row_b = static_cast<int64_t>(b) * L;
  const int64_t item0 = static_cast<int64_t>(bh) * chunks, kv0 = (static_cast<int64_t>(b) * G + kh) * chunks;
  const int64_t sb = (static_cast<int64_t>(bh) * P + (col_ok ? col : 0)) * N;
  const uint32_t yrow = static_cast<uint32_t>(H * P);
  // Byte offset of element (4 g, col) of a chunk of dY or dV; past any buffer where there is no column.
  const uint32_t ybase = col_ok ? (static_cast<uint32_t>(4 * g) * yrow + static_cast<uint32_t>(col)) * 4 : 0x80000000u;

  _Float16* const xh = reinterpret_cast<_Float16*>(xch[pr]);
  float* const xf = reinterpret_cast<float*>(xh + W::kXH);
  float *const xx_f = xf + W::kFS, *const xu_f = xx_f + 128, *const xb_f = xx_f + 192;
  const auto piece = [&](int at, int q, int half) __attribute__((always_inline)) {
    return reinterpret_cast<half8_t*>(xh + at + (2 * q + half) * kGdrFragHalves + lane * 8);
  };
  const auto ftile = [&](int at, int t) __attribute__((always_inline)) {
    return reinterpret_cast<f32x4_t*>(xf + at + t * 256 + lane * 4);
  };

  // Step `step` walks chunk n_chunks - 1 - step. Its phases end with barriers:
  // U is there (and T); kf dE and Q^T (qf dY) are there (and the next chunk's
  // factors); X' and the next Pm^T dY are there. With one buffer for K
  // it comes in behind the third, before a fourth.
  if (w < 2 * NPAIR) {
    // ---------------------------------------------------------------- X
    const int n0 = r * (NP / 2);
    f32x4_t X[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
        X[j][i] = (a.dh_final != nullptr && col_ok && n < N) ? flip(a.dh_final[sb + n], odd) : 0.0f;
      }
    }
    half8_t Xh[NK], Xl[NK];
    float x_down = 0.0f, xtop = 0.0f;
    auto split = [&]() __attribute__((always_inline)) {
      xtop = tiles_absmax<NJ>(X);
      const Pow2 s = pow2_to_top(xtop);
      x_down = s.down;
#pragma unroll
      for (int q = 0; q < NK; ++q) {
        tiles_to_operand<true>(X[2 * q], X[2 * q + 1], s.up, Xh[q], Xl[q]);
        *piece(W::kXX, r * NK + q, 0) = Xh[q];
        *piece(W::kXX, r * NK + q, 1) = Xl[q];
      }
      xx_f[64 * r + lane] = s.down;
    };
    split();
    __syncthreads();
    __syncthreads();

    for (int step = 0; step < n_chunks; ++step) {
      const int c = n_chunks - 1 - step;
      const _Float16* sK = reinterpret_cast<const _Float16*>(lds[W::NBUF == 2 ? (step & 1) : 0]);
      const float* sF = sFac[step & 1];
      const auto factor = [&](int which, int u) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x4_t*>(sF + which * kGdrC + 32 * r + 16 * u + 4 * g);
      };
      const int64_t item = item0 + c;
      float* const tops = ws.top + item * kGdrMaxima * kGdrMaxSlots + col / 16 * 2 + r;
      // U = Pm^T dY + diag(w) K X on the wave's 32 steps
      half8_t Uh, Ul;
      Pow2 su;
      {
        f32x4_t kx[2][2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
#pragma unroll
          for (int u = 0; u < 2; ++u) kx[o][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < NK; ++q) {
            const int f = (o == 0 ? r : 1 - r) * NK + q;
            const half8_t vh = o == 0 ? Xh[q] : *piece(W::kXX, f, 0);
            const half8_t vl = o == 0 ? Xl[q] : *piece(W::kXX, f, 1);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int at = kq_at<NP>(32 * r + 16 * u + m, 32 * f + 8 * g);
              const half8_t k = *reinterpret_cast<const half8_t*>(sK + at);
              kx[o][u] = mfma16(k, vh, kx[o][u]);
              kx[o][u] = mfma16(k, vl, kx[o][u]);
              if constexpr (RAW == 2) kx[o][u] = mfma16(*reinterpret_cast<const half8_t*>(sK + kLo + at), vh, kx[o][u]);
            }
          }
        }
        const float xo_down = xx_f[64 * (1 - r) + lane];
        f32x4_t U[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4_t fw = factor(2, u), py = *ftile(W::kFY, 2 * r + u);
#pragma unroll
          for (int i = 0; i < 4; ++i) U[u][i] = fmaf(fw[i], fmaf(kx[1][u][i], xo_down, kx[0][u][i] * x_down), py[i]);
        }
        su = pow2_to_top(tiles_absmax<2>(U));
        tiles_to_operand<true>(U[0], U[1], su.up, Uh, Ul);
        if (r == 1) {
          *piece(W::kXU, 0, 0) = Uh;
          *piece(W::kXU, 0, 1) = Ul;
          xu_f[lane] = su.down;
        }
      }
      if (col_ok) {
        float* dst = ws.X + (item * P + col) * N;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1);
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
      const float mx = lanes16_max(xtop);
      if (lane == 0 && col < P) tops[kMaxX * kGdrMaxSlots] = mx;
      __syncthreads();

      // dE = T^T U
      f32x4_t E[2];
      {
        const float tri = flip(sF[4 * kGdrC + 1], odd), down = su.down * tri;
        const auto T = [&](int f, int half) __attribute__((always_inline)) {
          return *reinterpret_cast<const half8_t*>(sT + (2 * f + half) * kGdrFragHalves + lane * 8);
        };
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int f = r == 0 ? 2 * u : 4 + u;
          const half8_t th = T(f, 0), tl = T(f, 1);
          f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          acc = mfma16(th, Uh, acc);
          acc = mfma16(th, Ul, acc);
          acc = mfma16(tl, Uh, acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) E[u][i] = acc[i] * down;
        }
        if (r == 0) {
          const half8_t oh = *piece(W::kXU, 0, 0), ol = *piece(W::kXU, 0, 1);
          const float other = xu_f[lane] * tri;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const half8_t th = T(2 * u + 1, 0), tl = T(2 * u + 1, 1);
            f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            acc = mfma16(th, oh, acc);
            acc = mfma16(th, ol, acc);
            acc = mfma16(tl, oh, acc);
#pragma unroll
            for (int i = 0; i < 4; ++i) E[u][i] = fmaf(acc[i], other, E[u][i]);
          }
        }
      }
      // kf dE as an operand for both waves
      half8_t Bh, Bl;
      Pow2 sd;
      {
        f32x4_t B[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4_t fk = factor(0, u);
#pragma unroll
          for (int i = 0; i < 4; ++i) B[u][i] = E[u][i] * -fk[i];
        }
        sd = pow2_to_top(tiles_absmax<2>(B));
        tiles_to_operand<true>(B[0], B[1], flip(sd.up, odd), Bh, Bl);
        *piece(W::kXB, r, 0) = Bh;
        *piece(W::kXB, r, 1) = Bl;
        xb_f[64 * r + lane] = sd.down;
      }
      const float end = sF[4 * kGdrC];
      __syncthreads();

      // X' = e^(c_end) X + Q^T (qf dY) - K^T (kf dE) on the wave's half of the rows
      {
        const half8_t oh = *piece(W::kXB, 1 - r, 0), ol = *piece(W::kXB, 1 - r, 1);
        const float d_own = sd.down, d_oth = xb_f[64 * (1 - r) + lane];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          f32x4_t acc[2];
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            acc[o] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            const half8_t bh = o == 0 ? Bh : oh, bl = o == 0 ? Bl : ol;
            const int at = kq_at<NP>(32 * (o == 0 ? r : 1 - r) + 4 * g + (m >> 2), n0 + 32 * (j / 2) + 8 * (m & 3)) + 4 * (j & 1);
            const auto column = [&](const _Float16* mat) __attribute__((always_inline)) {
              return __builtin_shufflevector(lds_column4(mat + at), lds_column4(mat + at + 16 * NP), 0, 1, 2, 3, 4, 5, 6, 7);
            };
            const half8_t kc = column(sK);
            acc[o] = mfma16(kc, bh, acc[o]);
            acc[o] = mfma16(kc, bl, acc[o]);
            if constexpr (RAW == 2) acc[o] = mfma16(column(sK + kLo), bh, acc[o]);
          }
          const f32x4_t qa = *ftile(W::kFQ, r * NJ + j);
#pragma unroll
          for (int i = 0; i < 4; ++i) X[j][i] = fmaf(acc[1][i], d_oth, fmaf(acc[0][i], d_own, fmaf(end, X[j][i], qa[i])));
        }
      }
      if (step + 1 < n_chunks) split();
      {
        const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
        const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
        const int out_rows = static_cast<int>(L - t0 < kGdrC ? L - t0 : kGdrC);
        const rsrc_t rv = rows_buffer<4>(a.dv, (row_b + t0) * yrow + static_cast<int64_t>(h) * P, out_rows, yrow, P);
        const float me = lanes16_max(tiles_absmax<2>(E));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = 32 * r + 16 * (i / 4) + (i % 4);
          buffer_store_f32<false>(t + 4 * g < rows ? E[i / 4][i % 4] : 0.0f, rv, ybase + static_cast<uint32_t>(t) * yrow * 4);
        }
        if (lane == 0 && col < P) tops[kMaxDE * kGdrMaxSlots] = me;
      }
      __syncthreads();
      if constexpr (W::NBUF == 1) __syncthreads();
    }
    if (a.dh0 != nullptr && col_ok) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
          if (n < N) a.dh0[sb + n] = flip(X[j][i], odd);
        }
      }
    }
    return;
  }

  // -------------------------------------------- loads, Pm^T dY and Q^T (qf dY)
  const int ltid = tid - 128 * NPAIR;
  const int n0 = r * (NP / 2);
  u32x4_t kr[W::NKQ], qr[W::NKQ], tr[W::NTL];
  float fr[W::NFL], yr[16];
  f32x2_t fe;
  half8_t Pd[2][2], Po[2][2], Ah[2], Al[2];
  float a_down = 0.0f;
  // (A load in no branch: it would be waited for where the branches join. No store
  // either: loads are counted from the last access backwards.)
  auto fetch_kq = [&](int c) __attribute__((always_inline)) {
    const u32x4_t* K = reinterpret_cast<const u32x4_t*>(ws.K + (kv0 + c) * W::kMat) + ltid;
    const u32x4_t* Q = reinterpret_cast<const u32x4_t*>(ws.Q + (kv0 + c) * W::kMat) + ltid;
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      kr[i] = K[i * W::NL];
      qr[i] = Q[i * W::NL];
    }
  };
  auto fetch_T = [&](int c) __attribute__((always_inline)) {
    const u32x4_t* T = reinterpret_cast<const u32x4_t*>(ws.Tt + (item0 + c) * kGdrPieceHalves) + ltid;
#pragma unroll
    for (int i = 0; i < W::NTL; ++i) tr[i] = T[i * W::NL];
  };
  auto fetch_fac = [&](int c) __attribute__((always_inline)) {
    const float* fac = ws.fac + (item0 + c) * (kGdrFactors * kGdrC);
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) fr[i] = fac[kFacK * kGdrC + (i * W::NL + ltid) % (4 * kGdrC)];
    fe = *reinterpret_cast<const f32x2_t*>(fac + kFacEnd * kGdrC);
  };
  // dY's rows, and the pieces of Pm^T for row tiles 2 r, 2 r + 1.
  auto fetch_y = [&](int c) __attribute__((always_inline)) {
    const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
    const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
    const rsrc_t ry = rows_buffer<4>(a.dy, (row_b + t0) * yrow + static_cast<int64_t>(h) * P, rows, yrow, P);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      yr[i] = __uint_as_float(buffer_load_bits<false>(ry, ybase + static_cast<uint32_t>(16 * (i / 4) + (i % 4)) * yrow * 4));
    }
    const half8_t* src = reinterpret_cast<const half8_t*>(ws.Pt + (item0 + c) * kGdrPieceHalves) + lane;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int fd = r == 0 ? 2 * u : 4 + u, fo = r == 0 ? 2 * u + 1 : fd;  // (wave 1 has no other: its own again)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Pd[u][k] = src[(2 * fd + k) * 64];
        Po[u][k] = src[(2 * fo + k) * 64];
      }
    }
  };
  auto stage_k = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) reinterpret_cast<u32x4_t*>(lds[buf])[i * W::NL + ltid] = kr[i];
  };
  auto stage_q = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) reinterpret_cast<u32x4_t*>(sQ)[i * W::NL + ltid] = qr[i];
  };
  auto stage_T = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W::NTL; ++i) reinterpret_cast<u32x4_t*>(sT)[i * W::NL + ltid] = tr[i];
  };
  auto stage_fac = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * W::NL + ltid;
      if (4 * kGdrC % W::NL == 0 || e < 4 * kGdrC) sFac[buf][e] = fr[i];
    }
    if (ltid == 0) *reinterpret_cast<f32x2_t*>(&sFac[buf][4 * kGdrC]) = fe;
  };
  // Pm^T dY of chunk c into LDS, qf dY as an operand into registers.
  auto from_y = [&](int c, int buf) __attribute__((always_inline)) {
    const float* sF = sFac[buf];
    f32x4_t Y[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) Y[i / 4][i % 4] = yr[i];
    const float ytop = tiles_absmax<4>(Y);
    const Pow2 sy = pow2_to_top(ytop);
    half8_t Yh[2], Yl[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) tiles_to_operand<true>(Y[2 * q], Y[2 * q + 1], flip(sy.up, odd), Yh[q], Yl[q]);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      const half8_t oh = r == 0 ? Yh[0] : Yh[1], ol = r == 0 ? Yl[0] : Yl[1];
      acc = mfma16(Pd[u][0], oh, acc);
      acc = mfma16(Pd[u][0], ol, acc);
      acc = mfma16(Pd[u][1], oh, acc);
      if (r == 0) {
        acc = mfma16(Po[u][0], Yh[1], acc);
        acc = mfma16(Po[u][0], Yl[1], acc);
        acc = mfma16(Po[u][1], Yh[1], acc);
      }
      const f32x4_t fp = *reinterpret_cast<const f32x4_t*>(sF + 3 * kGdrC + 32 * r + 16 * u + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= fp[i] * sy.down;
      *ftile(W::kFY, 2 * r + u) = acc;
    }
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      const f32x4_t fq = *reinterpret_cast<const f32x4_t*>(sF + 1 * kGdrC + 16 * tt + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) Y[tt][i] *= fq[i];
    }
    const Pow2 sa = pow2_to_top(tiles_absmax<4>(Y));
    a_down = sa.down;
#pragma unroll
    for (int q = 0; q < 2; ++q) tiles_to_operand<true>(Y[2 * q], Y[2 * q + 1], flip(sa.up, odd), Ah[q], Al[q]);
    const float my = lanes16_max(ytop);
    buffer_store_f32<false>(my, raw_buffer(ws.top + (item0 + c) * kGdrMaxima * kGdrMaxSlots, kGdrMaxima * kGdrMaxSlots * 4),
                            lane == 0 && col < P ? static_cast<uint32_t>(kMaxDY * kGdrMaxSlots + col / 16 * 2 + r) * 4 : kOutOfRange);
  };
  const auto chunk_at = [&](int step) { return step < n_chunks ? n_chunks - 1 - step : 0; };
  if (n_chunks > 0) {
    fetch_fac(chunk_at(0));
    fetch_kq(chunk_at(0));
    fetch_y(chunk_at(0));
    fetch_T(chunk_at(0));
    stage_fac(0);
    stage_k(0);
    stage_q();
    fetch_fac(chunk_at(1));
    fetch_kq(chunk_at(1));
  }
  __syncthreads();  // (the factors, for the first Pm^T dY)
  if (n_chunks > 0) {
    from_y(chunk_at(0), 0);
    fetch_y(chunk_at(1));
  }
  __syncthreads();
  for (int step = 0; step < n_chunks; ++step) {
    stage_T();
    // Q^T (qf dY) on half r of the rows of X
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int at = kq_at<NP>(32 * q + 4 * g + (m >> 2), n0 + 32 * (j / 2) + 8 * (m & 3)) + 4 * (j & 1);
        const auto column = [&](const _Float16* mat) __attribute__((always_inline)) {
          return __builtin_shufflevector(lds_column4(mat + at), lds_column4(mat + at + 16 * NP), 0, 1, 2, 3, 4, 5, 6, 7);
        };
        const half8_t qc = column(sQ);
        acc = mfma16(qc, Ah[q], acc);
        acc = mfma16(qc, Al[q], acc);
        if constexpr (RAW == 2) acc = mfma16(column(sQ + kLo), Ah[q], acc);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= a_down;
      *ftile(W::kFQ, r * NJ + j) = acc;
    }
    __syncthreads();
    stage_fac((step + 1) & 1);
    fetch_fac(chunk_at(step + 2));
    stage_q();
    if constexpr (W::NBUF == 2) {
      stage_k((step + 1) & 1);
      fetch_kq(chunk_at(step + 2));
    }
    fetch_T(chunk_at(step + 1));
    __syncthreads();
    if (step + 1 < n_chunks) from_y(chunk_at(step + 1), (step + 1) & 1);
    fetch_y(chunk_at(step + 2));
    __syncthreads();
    if constexpr (W::NBUF == 1) {
      stage_k(0);
      fetch_kq(chunk_at(step + 2));
      __syncthreads();
    }
  }
  for (int64_t t = static_cast<int64_t>(n_chunks) * kGdrC + 4 * r + g; t < L; t += 8) {
    if (col_ok) a.dv[(row_b + t) * yrow + static_cast<int64_t>(h) * P + col] = 0.0f;
  }
}

template <int NP, bool BF16, int NPAIR>
__global__ __launch_bounds__(256 * NPAIR) void gdr_reverse_kernel(const GatedDeltaBwdArgs a, const GdrWork ws, int chunks) {
  __shared__ GdrBackLds<GdrBack<NP, BF16, NPAIR>, NPAIR> lds;
  gdr_walk_back<NP, BF16, NPAIR>(a, ws, chunks, static_cast<int>(blockIdx.x), static_cast<int>(threadIdx.x), lds);
}

// Both walks of a slice at once, forth by the first four waves and back by the
// others: neither needs anything of the other. They share the barriers, of which
// the walk back has one more in front. (2, 4096, 16 heads of 128 x 128, bfloat16):
// 260 us now; when it was built 295 where the two kernels took 327, and with half
// the batch 257 us for the whole backward in place of 335.
template <int NP, bool BF16>
__global__ __launch_bounds__(512) void gdr_both_kernel(const GatedDeltaBwdArgs a, const GdrWork ws, int chunks) {
  using Forth = GdrWalk<NP, BF16, true, 1, kGdrKeep>;
  using Back = GdrBack<NP, BF16, 1>;
  static_assert(Forth::NT == 256 && Forth::NBUF == 2 && !Forth::kLag && Back::NBUF == 2);
  __shared__ GdrWalkLds<Forth, 1> forth;
  __shared__ GdrBackLds<Back, 1> back;
  static_assert(sizeof(forth) + sizeof(back) <= 160 * 1024);
  const int tid = static_cast<int>(threadIdx.x);
  if (__builtin_amdgcn_readfirstlane(tid >> 8) == 0) {
    __syncthreads();
    gdr_walk<NP, BF16, true, 1, kGdrKeep>(a.f, ws, chunks, 1, chunks, static_cast<int>(blockIdx.x), tid, forth);
  } else {
    gdr_walk_back<NP, BF16, 1>(a, ws, chunks, static_cast<int>(blockIdx.x), (tid - 256) ^ 128, back);
  }
}

template <int NP, bool BF16>
void launch_pairs(const GatedDeltaBwdArgs& a, const GdrWork& ws, int chunks, hipStream_t st) {
  const int64_t bh = a.f.batch * a.f.nheads;
  const int64_t slices = (a.f.headdim + 15) / 16;
  const unsigned one = static_cast<unsigned>(bh * slices);
  if (gdr_block_pairs(bh, slices) > 1) {
    gdr_reverse_kernel<NP, BF16, 2><<<static_cast<unsigned>(bh * ((slices + 1) / 2)), 512, 0, st>>>(a, ws, chunks);
  } else if constexpr (gdr_both_fit(NP, BF16)) {
    gdr_both_kernel<NP, BF16><<<one, 512, 0, st>>>(a, ws, chunks);
  } else {
    gdr_reverse_kernel<NP, BF16, 1><<<one, 256, 0, st>>>(a, ws, chunks);
  }
}

}  // namespace

int launch_gdr_reverse(const GatedDeltaBwdArgs& a, const GdrWork& ws, int64_t chunks, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int n = static_cast<int>(chunks);
  const auto width = [&](auto np) {
    constexpr int NP = decltype(np)::value;
    a.f.in_bf16 ? launch_pairs<NP, true>(a, ws, n, st) : launch_pairs<NP, false>(a, ws, n, st);
  };
  if (a.f.dstate <= 64) {
    width(std::integral_constant<int, 64>{});
  } else {
    width(std::integral_constant<int, 128>{});
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
