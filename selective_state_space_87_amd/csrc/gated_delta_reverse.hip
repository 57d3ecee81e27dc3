// Gated delta rule backward, the walk back over a head's chunks (see gdr_mma.h).
// With the gradient X of the state leaving a chunk, dY the output's:
//   U  = Pm^T dY + diag(w) K X            (of E, as the later ones see it)
//   dE = T^T U                            (of V - diag(e^c) K S; also dV)
//   X' = e^(c_end) X + Q^T (qf dY) - K^T (kf dE)
// the mirror image of the forward's walk, and split the same way: a pair of
// waves owns 16 columns of X in registers; wave r takes steps 32 r .. + 31 of
// the first two lines and half r of the N rows of the third. Through LDS go X
// (both ways), dY and U of the last 32 steps (to the wave of the first), and
// the third line's operands. X is left in the workspace for every chunk (the
// gradient of its leaving state), dE in dv.
#include <hip/hip_runtime.h>

#include "gdr_mma.h"

namespace ssm {

namespace {

template <int NP, bool BF16, int NPAIR>
struct GdrBack {
  static constexpr int NT = 128 * NPAIR;
  static constexpr int RAW = BF16 ? 1 : 2;
  static constexpr int kMat = RAW * kGdrC * NP;
  static constexpr int kFac = 4 * kGdrC;                // K, Q, W, P factors
  static constexpr int kBufBytes = 2 * kMat * 2 + kFac * 4;
  // a pair's exchange, in halves: X (NP / 32 pieces), dY, U, (qf dY and kf dE of either wave); then scales
  static constexpr int kXX = 0, kXY = kXX + NP / 32 * 2 * kGdrFragHalves, kXU = kXY + 2 * kGdrFragHalves;
  static constexpr int kXD = kXU + 2 * kGdrFragHalves, kXF = kXD + 8 * kGdrFragHalves;
  static constexpr int kPairBytes = kXF * 2 + 6 * 64 * 4;
  static constexpr int NBUF = 2 * kBufBytes + NPAIR * kPairBytes <= 160 * 1024 ? 2 : 1;
  static constexpr int NKQ = kMat / 8 / NT;
  static constexpr int NFL = (4 * kGdrC + NT - 1) / NT;
};

template <int NP, bool BF16, int NPAIR>
__global__ __launch_bounds__(128 * NPAIR, NPAIR == 4 ? 2 : 1) void gdr_reverse_kernel(const GatedDeltaBwdArgs a,
                                                                                      const GdrWork ws, int chunks) {
  using W = GdrBack<NP, BF16, NPAIR>;
  constexpr int NT = W::NT, RAW = W::RAW, NJ = NP / 32, NK = NP / 64;
  constexpr int kLo = kGdrC * NP;
  __shared__ __align__(16) char lds[W::NBUF][W::kBufBytes];
  __shared__ __align__(16) char xch[NPAIR][W::kPairBytes];
  const GatedDeltaArgs& p = a.f;

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
  float *const xx_f = xf, *const xy_f = xf + 128, *const xu_f = xf + 192, *const xd_f = xf + 256;
  const auto piece = [&](int at, int q, int half) __attribute__((always_inline)) {
    return reinterpret_cast<half8_t*>(xh + at + (2 * q + half) * kGdrFragHalves + lane * 8);
  };

  const int n0 = r * (NP / 2);
  f32x4_t X[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
      X[j][i] = (a.dh_final != nullptr && col_ok && n < N) ? a.dh_final[sb + n] : 0.0f;
    }
  }

  u32x4_t kr[W::NKQ], qr[W::NKQ];
  float fr[W::NFL], yr[8];
  float fend = 0.0f, ftri = 0.0f, fend_next = 0.0f, ftri_next = 0.0f;
  half8_t Td[2][2], To[2][2], Pd[2][2], Po[2][2];  // pieces on the diagonal, and right of it (wave 0)

  // (No load of the next chunk stands in a branch: it would be waited for
  // where the branches join.)
  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
    const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
    const rsrc_t ry = rows_buffer<4>(a.dy, (row_b + t0) * yrow + static_cast<int64_t>(h) * P, rows, yrow, P);
    const float* fac = ws.fac + (item0 + c) * (kGdrFactors * kGdrC);
    const u32x4_t* K = reinterpret_cast<const u32x4_t*>(ws.K + (kv0 + c) * W::kMat) + tid;
    const u32x4_t* Q = reinterpret_cast<const u32x4_t*>(ws.Q + (kv0 + c) * W::kMat) + tid;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = 32 * r + 16 * (i / 4) + 4 * g + (i % 4);
      const uint32_t off = (static_cast<uint32_t>(t) * yrow + static_cast<uint32_t>(col)) * 4;
      yr[i] = __uint_as_float(buffer_load_bits<false>(ry, col_ok ? off : kOutOfRange));
    }
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      kr[i] = K[i * NT];
      qr[i] = Q[i * NT];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * NT + tid;
      fr[i] = fac[kFacK * kGdrC + (4 * kGdrC % NT == 0 ? e : e % (4 * kGdrC))];
    }
    fend_next = fac[kFacEnd * kGdrC];
    ftri_next = fac[kFacEnd * kGdrC + 1];
  };
  auto fetch_tri = [&](const _Float16* base, int c, half8_t (&d)[2][2], half8_t (&o)[2][2])
                       __attribute__((always_inline)) {
    const half8_t* src = reinterpret_cast<const half8_t*>(base + (item0 + c) * kGdrPieceHalves) + lane;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int fd = r == 0 ? 2 * u : 4 + u, fo = r == 0 ? 2 * u + 1 : fd;  // (wave 1 has no other: its own again)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        d[u][k] = src[(2 * fd + k) * 64];
        o[u][k] = src[(2 * fo + k) * 64];
      }
    }
  };
  auto stage = [&](int buf) __attribute__((always_inline)) {
    _Float16* sK = reinterpret_cast<_Float16*>(lds[buf]);
    _Float16* sQ = sK + W::kMat;
    float* sF = reinterpret_cast<float*>(sQ + W::kMat);
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      reinterpret_cast<u32x4_t*>(sK)[i * NT + tid] = kr[i];
      reinterpret_cast<u32x4_t*>(sQ)[i * NT + tid] = qr[i];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * NT + tid;
      if (4 * kGdrC % NT == 0 || e < 4 * kGdrC) sF[e] = fr[i];
    }
    fend = fend_next;
    ftri = ftri_next;
  };

  half8_t Xh[NK], Xl[NK], Yh, Yl;
  f32x4_t Y[2];
  float x_down = 0.0f, y_down = 0.0f, xtop = 0.0f, ytop = 0.0f;
  // X and the next chunk's dY as operands, for this wave and for the other.
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
#pragma unroll
    for (int i = 0; i < 8; ++i) Y[i / 4][i % 4] = yr[i];
    ytop = tiles_absmax<2>(Y);
    const Pow2 sy = pow2_to_top(ytop);
    y_down = sy.down;
    tiles_to_operand<true>(Y[0], Y[1], sy.up, Yh, Yl);
    if (r == 1) {
      *piece(W::kXY, 0, 0) = Yh;
      *piece(W::kXY, 0, 1) = Yl;
      xy_f[lane] = sy.down;
    }
  };

  if (n_chunks > 0) {
    fetch(n_chunks - 1);
    fetch_tri(ws.Tt, n_chunks - 1, Td, To);
    fetch_tri(ws.Pt, n_chunks - 1, Pd, Po);
    stage(0);
    split();
  }
  __syncthreads();

  for (int step = 0; step < n_chunks; ++step) {
    const int c = n_chunks - 1 - step;
    const int buf = W::NBUF == 2 ? (step & 1) : 0;
    const _Float16* sK = reinterpret_cast<const _Float16*>(lds[buf]);
    const _Float16* sQ = sK + W::kMat;
    const float* sF = reinterpret_cast<const float*>(sQ + W::kMat);
    const auto factor = [&](int which, int u) __attribute__((always_inline)) {
      return *reinterpret_cast<const f32x4_t*>(sF + which * kGdrC + 32 * r + 16 * u + 4 * g);
    };
    const bool more = c > 0;
    const int next = more ? c - 1 : 0;
    fetch(next);

    const int64_t item = item0 + c;
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

    // U = Pm^T dY + diag(w) K X on the wave's 32 steps
    half8_t Uh, Ul;
    Pow2 su;
    {
      f32x4_t kx[2][2], py[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) kx[0][u] = kx[1][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int o = 0; o < 2; ++o) {
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
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        acc = mfma16(Pd[u][0], Yh, acc);
        acc = mfma16(Pd[u][0], Yl, acc);
        acc = mfma16(Pd[u][1], Yh, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) py[u][i] = acc[i] * y_down;
      }
      if (r == 0) {
        const half8_t oh = *piece(W::kXY, 0, 0), ol = *piece(W::kXY, 0, 1);
        const float other = xy_f[lane];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          acc = mfma16(Po[u][0], oh, acc);
          acc = mfma16(Po[u][0], ol, acc);
          acc = mfma16(Po[u][1], oh, acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) py[u][i] = fmaf(acc[i], other, py[u][i]);
        }
      }
      fetch_tri(ws.Pt, next, Pd, Po);
      const float xo_down = xx_f[64 * (1 - r) + lane];
      f32x4_t U[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4_t fw = factor(2, u), fp = factor(3, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          U[u][i] = fmaf(fw[i], fmaf(kx[1][u][i], xo_down, kx[0][u][i] * x_down), fp[i] * py[u][i]);
        }
      }
      su = pow2_to_top(tiles_absmax<2>(U));
      tiles_to_operand<true>(U[0], U[1], su.up, Uh, Ul);
      if (r == 1) {
        *piece(W::kXU, 0, 0) = Uh;
        *piece(W::kXU, 0, 1) = Ul;
        xu_f[lane] = su.down;
      }
    }
    __syncthreads();

    // dE = T^T U
    f32x4_t E[2];
    {
      const float down = su.down * ftri;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        acc = mfma16(Td[u][0], Uh, acc);
        acc = mfma16(Td[u][0], Ul, acc);
        acc = mfma16(Td[u][1], Uh, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) E[u][i] = acc[i] * down;
      }
      if (r == 0) {
        const half8_t oh = *piece(W::kXU, 0, 0), ol = *piece(W::kXU, 0, 1);
        const float other = xu_f[lane] * ftri;
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
    fetch_tri(ws.Tt, next, Td, To);
    // qf dY and -kf dE as operands for both waves, one scale for the two so that one accumulator takes them
    half8_t Ah, Al, Bh, Bl;
    Pow2 sd;
    {
      f32x4_t A[2], B[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4_t fk = factor(0, u), fq = factor(1, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          A[u][i] = Y[u][i] * fq[i];
          B[u][i] = E[u][i] * -fk[i];
        }
      }
      sd = pow2_to_top(fmaxf(tiles_absmax<2>(A), tiles_absmax<2>(B)));
      tiles_to_operand<true>(A[0], A[1], sd.up, Ah, Al);
      tiles_to_operand<true>(B[0], B[1], sd.up, Bh, Bl);
      *piece(W::kXD, 2 * r, 0) = Ah;
      *piece(W::kXD, 2 * r, 1) = Al;
      *piece(W::kXD, 2 * r + 1, 0) = Bh;
      *piece(W::kXD, 2 * r + 1, 1) = Bl;
      xd_f[64 * r + lane] = sd.down;
    }
    __syncthreads();

    // X' = e^(c_end) X + Q^T (qf dY) - K^T (kf dE) on the wave's half of the rows
    {
      const half8_t oah = *piece(W::kXD, 2 * (1 - r), 0), oal = *piece(W::kXD, 2 * (1 - r), 1);
      const half8_t obh = *piece(W::kXD, 2 * (1 - r) + 1, 0), obl = *piece(W::kXD, 2 * (1 - r) + 1, 1);
      const float d_own = sd.down, d_oth = xd_f[64 * (1 - r) + lane];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        f32x4_t acc[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          acc[o] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          const half8_t vah = o == 0 ? Ah : oah, val = o == 0 ? Al : oal, vbh = o == 0 ? Bh : obh, vbl = o == 0 ? Bl : obl;
          const int at = kq_at<NP>(32 * (o == 0 ? r : 1 - r) + 4 * g + (m >> 2), n0 + 32 * (j / 2) + 8 * (m & 3)) + 4 * (j & 1);
          const auto column = [&](const _Float16* mat) __attribute__((always_inline)) {
            return __builtin_shufflevector(lds_column4(mat + at), lds_column4(mat + at + 16 * NP), 0, 1, 2, 3, 4, 5, 6, 7);
          };
          const half8_t kc = column(sK), qc = column(sQ);
          acc[o] = mfma16(qc, vah, acc[o]);
          acc[o] = mfma16(qc, val, acc[o]);
          acc[o] = mfma16(kc, vbh, acc[o]);
          acc[o] = mfma16(kc, vbl, acc[o]);
          if constexpr (RAW == 2) {
            acc[o] = mfma16(column(sQ + kLo), vah, acc[o]);
            acc[o] = mfma16(column(sK + kLo), vbh, acc[o]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) X[j][i] = fmaf(acc[1][i], d_oth, fmaf(acc[0][i], d_own, fend * X[j][i]));
      }
    }
    {
      const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
      const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
      const int out_rows = static_cast<int>(L - t0 < kGdrC ? L - t0 : kGdrC);
      const rsrc_t rv = rows_buffer<4>(a.dv, (row_b + t0) * yrow + static_cast<int64_t>(h) * P, out_rows, yrow, P);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = 32 * r + 16 * (i / 4) + 4 * g + (i % 4);
        const uint32_t off = (static_cast<uint32_t>(t) * yrow + static_cast<uint32_t>(col)) * 4;
        buffer_store_f32<false>(t < rows ? E[i / 4][i % 4] : 0.0f, rv, col_ok ? off : kOutOfRange);
      }
      const float mx = lanes16_max(xtop), my = lanes16_max(ytop), me = lanes16_max(tiles_absmax<2>(E));
      if (lane == 0 && col < P) {
        float* top = ws.top + item * kGdrMaxima * kGdrMaxSlots + col / 16 * 2 + r;
        top[kMaxX * kGdrMaxSlots] = mx;
        top[kMaxDY * kGdrMaxSlots] = my;
        top[kMaxDE * kGdrMaxSlots] = me;
      }
    }
    if (more) split();
    if constexpr (W::NBUF == 1) __syncthreads();
    if (more) stage(W::NBUF == 2 ? ((step + 1) & 1) : 0);
    __syncthreads();
  }

  for (int64_t t = static_cast<int64_t>(n_chunks) * kGdrC + 4 * r + g; t < L; t += 8) {
    if (col_ok) a.dv[(row_b + t) * yrow + static_cast<int64_t>(h) * P + col] = 0.0f;
  }
  if (a.dh0 != nullptr && col_ok) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
        if (n < N) a.dh0[sb + n] = X[j][i];
      }
    }
  }
}

template <int NP, bool BF16>
void launch_pairs(const GatedDeltaBwdArgs& a, const GdrWork& ws, int chunks, hipStream_t st) {
  const int64_t bh = a.f.batch * a.f.nheads;
  const int64_t slices = (a.f.headdim + 15) / 16;
  const int pairs = gdr_block_pairs(bh, slices);
  const auto blocks = [&](int n) { return static_cast<unsigned>(bh * ((slices + n - 1) / n)); };
  if (pairs == 1) {
    gdr_reverse_kernel<NP, BF16, 1><<<blocks(1), 128, 0, st>>>(a, ws, chunks);
  } else if (pairs == 2) {
    gdr_reverse_kernel<NP, BF16, 2><<<blocks(2), 256, 0, st>>>(a, ws, chunks);
  } else {
    gdr_reverse_kernel<NP, BF16, 4><<<blocks(4), 512, 0, st>>>(a, ws, chunks);
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
