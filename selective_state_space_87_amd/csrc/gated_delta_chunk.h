// Gated delta rule, the walk over a head's chunks (see gdr_mma.h for the
// chunk's equations, operand halves and layouts). Included by one source file
// per input type.
//
// Sixteen columns of a head's state [N, P] belong to a pair of waves for the
// whole sequence. A chunk is a chain of products on them,
//   K S  ->  E = T (V - ..)  ->  S' = .. + K^T (w E)
// and the pair splits every link: of the products with K and T wave r of the
// pair takes the 32 steps 32 r .. + 31, of the state's update the half r of
// the N rows. What one needs of the other goes through LDS as the operand
// halves it is used as (S, R of the first 32 steps, and w E), three barriers a
// chunk. Everything that the next chunk does not wait for is taken off these
// waves: waves of their own read S and E from the exchange and form
//   Y = diag(scale e^c) Q S + Pm E
// one phase behind, and move K, Q, T, Pm and the factors of the next chunk from
// memory through their registers into LDS. Every product is of two halves, for a
// bfloat16 y too: with one in those of y, y is off by 2^-11 of its terms, which
// cancel, and the whole forward below took 568 us in place of 654.
// A chain as long as this is bound by what a single wave can issue, not by the
// units. Measured at (4, 8192, 16 key and 32 value heads of 128 x 128), bfloat16:
// 458 us, 3.6 us a chunk with four pairs a CU; vector instructions 52 % of a SIMD's
// cycles, LDS 55 %, matrix cores 29 %. (When it was built, against the walk of that
// time: one wave for all of a slice's work 790 us, a pair without waves for y and
// the loads 590, with them 520.)
#pragma once

#include "gdr_mma.h"

namespace ssm {

// What a walk is for: y; the backward's entering states and E, left in the
// workspace; or a segment's map (see gdr_segments.hip). The last two touch
// neither Q nor Pm.
enum GdrMode { kGdrForward, kGdrKeep, kGdrMap };

template <int NP, bool BF16, bool OB16, int NPAIR, int MODE>
struct GdrWalk {
  static constexpr bool KEEP = MODE != kGdrForward;
  static constexpr int RAW = BF16 ? 1 : 2;
  // Waves for y and the loads: one for every 32 steps of a slice. (KEEP with
  // four pairs: half as many, which have less to load; with sixteen waves a
  // wave's 128 registers would not do.)
  static constexpr int NOUT = KEEP && NPAIR == 4 ? 4 : 2 * NPAIR;
  static constexpr int kHalvesOut = 2 * NPAIR / NOUT;
  static constexpr int NT = 64 * (2 * NPAIR + NOUT);
  static constexpr int NL = 64 * NOUT;                  // threads that load
  static constexpr int kMat = RAW * kGdrC * NP;         // halves of K (or Q)
  static constexpr int kT = kGdrFrags * 2 * kGdrFragHalves;
  static constexpr int kP = KEEP ? 0 : kT;
  static constexpr int kFac = 4 * kGdrC + 4;            // K, Q, W, P factors; the end's and T's
  static constexpr int kBufBytes = (KEEP ? 1 : 2) * kMat * 2 + kFac * 4;
  // a pair's exchange, in halves: S (NP / 32 pieces), R of wave 0, w E (2), E of wave
  // 0; then scales (floats, a column each). E of wave 1 takes the place of R, which
  // that wave has read by then, and wave 0 writes again a barrier after E's last use.
  static constexpr int kXS = 0, kXR = kXS + NP / 32 * 2 * kGdrFragHalves, kXD = kXR + 2 * kGdrFragHalves;
  static constexpr int kXE = kXD + 4 * kGdrFragHalves, kXF = kXE + (KEEP ? 0 : 2 * kGdrFragHalves);
  static constexpr int kSS = 0, kSD = 32, kSE = 64, kSR = 96, kScales = 112;
  static constexpr int kPairBytes = kXF * 2 + kScales * 4;
  static constexpr int kFixed = (kT + kP) * 2 + NPAIR * kPairBytes;
  static constexpr int NBUF = 2 * kBufBytes + kFixed <= 160 * 1024 ? 2 : 1;
  // Four pairs (sixteen waves) have 128 registers a wave: enough with one half in
  // K and Q. Elsewhere two pairs.
  static constexpr bool kFits = NBUF * kBufBytes + kFixed <= 160 * 1024 && (KEEP || RAW == 1);
  // With two buffers, half the pairs run one phase behind the others.
  static constexpr bool kLag = NBUF == 2 && NPAIR >= 2;
  static constexpr int NKQ = kMat / 8 / NL;             // 16-byte pieces of K (and Q) a loading thread
  static constexpr int NTL = (kT / 8 + NL - 1) / NL;
  static constexpr int NPL = (kP / 8 + NL - 1) / NL;
  static constexpr int NFL = (4 * kGdrC + NL - 1) / NL;
};

// A walk's LDS.
template <class W, int NPAIR>
struct GdrWalkLds {
  __align__(16) char kq[W::NBUF][W::kBufBytes];
  __align__(16) _Float16 T[W::kT];
  __align__(16) _Float16 P[W::kP > 0 ? W::kP : 8];
  __align__(16) char xch[NPAIR][W::kPairBytes];
};

// The walk of block `block`, by threads 0 .. W::NT - 1 (tid). Its barriers: one,
// three a chunk (four with one buffer), and one more where pairs lag.
template <int NP, bool BF16, bool OB16, int NPAIR, int MODE>
__device__ __forceinline__ void gdr_walk(const GatedDeltaArgs& p, const GdrWork& ws, int chunks, int segs,
                                         int seg_chunks, int block, int tid,
                                         GdrWalkLds<GdrWalk<NP, BF16, OB16, NPAIR, MODE>, NPAIR>& sh) {
  using W = GdrWalk<NP, BF16, OB16, NPAIR, MODE>;
  constexpr bool KEEP = W::KEEP;
  constexpr int RAW = W::RAW;
  constexpr int kLo = kGdrC * NP;                       // from an element's hi half to its lo half
  constexpr int NJ = NP / 32, NK = NP / 64;             // state tiles and operand pieces of a wave
  constexpr int EB = BF16 ? 2 : 4;
  auto& lds = sh.kq;
  auto& xch = sh.xch;
  _Float16 *const sT = sh.T, *const sP = sh.P;

  const int lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads);
  const int N = static_cast<int>(p.dstate), P = static_cast<int>(p.headdim);
  const int cols = MODE == kGdrMap ? P + N : P;  // a map's columns: a state from zero, then the unit vectors
  const int pblocks = (cols + 16 * NPAIR - 1) / (16 * NPAIR);
  // K and Q are read by every slice of the heads that share them, T and Pm by every slice of a head.
  const int place = gdr_xcd_place(block, static_cast<int>(gridDim.x), segs == 1 ? H / G * pblocks : pblocks);
  const int walk_id = place / pblocks;
  const int bh = walk_id / segs, z = walk_id % segs;
  const int b = bh / H, h = bh % H, kh = h / (H / G);
  const int col0 = (place % pblocks) * 16 * NPAIR;
  // The segment: steps from `first` on, at most seg_chunks chunks.
  const int64_t first = static_cast<int64_t>(z) * seg_chunks * kGdrC, most = static_cast<int64_t>(seg_chunks) * kGdrC;
  const int64_t row_len = gdr_row_steps(p.seqlens, b, p.seqlen);
  const bool last_seg = row_len <= first + most && (row_len > first || z == 0);
  if (MODE == kGdrMap && (row_len <= first + most || (z == 0 && col0 >= P))) return;  // nothing follows; a known state
  const int64_t len = row_len <= first ? 0 : (row_len - first < most ? row_len - first : most);
  const int64_t L = p.seqlen - first < most ? p.seqlen - first : most;
  const int n_chunks = static_cast<int>((len + kGdrC - 1) / kGdrC);
  const int64_t row_b = static_cast<int64_t>(b) * p.seqlen + first;
  const int64_t item0 = static_cast<int64_t>(bh) * chunks + z * seg_chunks;
  const int64_t kv0 = (static_cast<int64_t>(b) * G + kh) * chunks + z * seg_chunks;
  const uint32_t yrow = static_cast<uint32_t>(H * P);

  // A phase ends with a barrier, three a chunk: R is there; w E and E are
  // there; S' is there. Pairs that lag take part in one barrier before their
  // first phase, the others in one behind their last. Into LDS go, counted in
  // phases of the pairs that do not lag: T of chunk c in phase 3 c (read from
  // 3 c + 1, last by the lagging pairs in 3 c + 2), Pm in 3 c + 1 (read in 3 c + 2
  // and 3 c + 3), K, Q and the factors of chunk c + 1 in 3 c + 1 and 3 c + 2, into
  // the buffer that was last read in 3 c. With one buffer nobody lags, and K, Q and
  // the factors come in between two barriers more, when the old ones are done with.
  if (w < 2 * NPAIR) {
    // ---------------------------------------------------------------- state
    const int pr = w >> 1, r = w & 1;
    const int col = col0 + 16 * pr + m;
    const bool col_ok = col < P;
    const int64_t sb = (static_cast<int64_t>(bh) * P + (col_ok ? col : 0)) * N;
    // (In segments, not from h0: another segment's block may write it as h_final.)
    const float* enters = p.h0;
    if (MODE == kGdrMap && z > 0) enters = nullptr;
    if (MODE == kGdrForward && segs > 1) enters = ws.seg + z * ws.seg_stride;
    _Float16* const xh = reinterpret_cast<_Float16*>(xch[pr]);
    float* const xf = reinterpret_cast<float*>(xh + W::kXF);
    float *const xs_f = xf + W::kSS + m, *const xd_f = xf + W::kSD + m, *const xe_f = xf + W::kSE + m, *const xr_f = xf + W::kSR + m;
    const auto piece = [&](int at, int q, int half) __attribute__((always_inline)) {
      return reinterpret_cast<half8_t*>(xh + at + (2 * q + half) * kGdrFragHalves + lane * 8);
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
        S[j][i] = (enters != nullptr && col_ok && n < N) ? enters[sb + n] : 0.0f;
        if (MODE == kGdrMap && col == P + n) S[j][i] = 1.0f;
      }
    }
    // The wave's rows of V, a chunk ahead. (No load of a next chunk stands in a
    // branch, here or below: it would be waited for where the branches join.)
    // (bfloat16 as 16 bits until it is used: carried in 32 it is masked every time.)
    std::conditional_t<BF16, uint16_t, uint32_t> vr[8];
    const uint32_t vs = static_cast<uint32_t>(p.v_step);
    const uint32_t vbase = col_ok ? (static_cast<uint32_t>(32 * r + 4 * g) * vs + static_cast<uint32_t>(col)) * EB : 0x80000000u;
    auto fetch_v = [&](int c) __attribute__((always_inline)) {
      const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
      const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
      const rsrc_t rv = rows_buffer<EB>(p.v, (row_b + t0) * p.v_step + static_cast<int64_t>(h) * P, rows, vs, P);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        vr[i] = static_cast<std::remove_reference_t<decltype(vr[i])>>(
            buffer_load_bits<BF16>(rv, vbase + static_cast<uint32_t>(16 * (i / 4) + (i % 4)) * vs * EB));
      }
    };

    half8_t Sh[NK], Sl[NK];
    float s_down = 0.0f, s_top = 0.0f;
    // The wave's half of S as an operand, for itself and for the others.
    auto split_S = [&]() __attribute__((always_inline)) {
      s_top = tiles_absmax<NJ>(S);
      const Pow2 s = pow2_to_top(s_top);
      s_down = s.down;
#pragma unroll
      for (int q = 0; q < NK; ++q) {
        tiles_to_operand<true>(S[2 * q], S[2 * q + 1], s.up, Sh[q], Sl[q]);
        *piece(W::kXS, r * NK + q, 0) = Sh[q];
        *piece(W::kXS, r * NK + q, 1) = Sl[q];
      }
      xs_f[16 * r] = s.down;
    };
    if (n_chunks > 0) fetch_v(0);
    split_S();
    const bool lag = W::kLag && pr >= NPAIR / 2;
    __syncthreads();
    if (lag) __syncthreads();

    for (int c = 0; c < n_chunks; ++c) {
      const int buf = W::NBUF == 2 ? (c & 1) : 0;
      const _Float16* sK = reinterpret_cast<const _Float16*>(lds[buf]);
      const float* sF = reinterpret_cast<const float*>(sK + (KEEP ? 1 : 2) * W::kMat);
      const auto factor = [&](int which, int u) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x4_t*>(sF + which * kGdrC + 32 * r + 16 * u + 4 * g);
      };
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (BF16) {
          v[i] = static_cast<float>(__builtin_bit_cast(__bf16, vr[i]));
        } else {
          v[i] = __uint_as_float(vr[i]);
        }
      }
      const bool more = c + 1 < n_chunks;
      fetch_v(more ? c + 1 : c);
      // (Stores in no branch either, here and for E: V's loads are counted from the
      // last access backwards, and behind a store that may have been skipped they
      // would be waited for with all stores.)
      if constexpr (MODE == kGdrKeep) {
        const int64_t item = item0 + c;
        const rsrc_t rs = raw_buffer(ws.S + item * P * N, static_cast<uint32_t>(P * N * 4));
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1);
          const uint32_t at = static_cast<uint32_t>(col * N + n) * 4;
          if (N % 4 == 0) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[j]), rs, col_ok && n < N ? at : kOutOfRange, 0, 0);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              buffer_store_f32<false>(S[j][i], rs, col_ok && n + i < N ? at + static_cast<uint32_t>(4 * i) : kOutOfRange);
            }
          }
        }
        buffer_store_f32<false>(lanes16_max(s_top), raw_buffer(ws.top + item * kGdrMaxima * kGdrMaxSlots, kGdrMaxima * kGdrMaxSlots * 4),
                                lane == 0 && col < P ? static_cast<uint32_t>(kMaxS * kGdrMaxSlots + col / 16 * 2 + r) * 4 : kOutOfRange);
      }

      // K S on the wave's 32 steps: its own half of S, and the other's.
      f32x4_t ks[2][2];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
#pragma unroll
        for (int u = 0; u < 2; ++u) ks[o][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < NK; ++q) {
          const int f = (o == 0 ? r : 1 - r) * NK + q;
          const half8_t sh = o == 0 ? Sh[q] : *piece(W::kXS, f, 0);
          const half8_t sl = o == 0 ? Sl[q] : *piece(W::kXS, f, 1);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int at = kq_at<NP>(32 * r + 16 * u + m, 32 * f + 8 * g);
            const half8_t a = *reinterpret_cast<const half8_t*>(sK + at);
            ks[o][u] = mfma16(a, sh, ks[o][u]);
            ks[o][u] = mfma16(a, sl, ks[o][u]);
            if constexpr (RAW == 2) {
              ks[o][u] = mfma16(*reinterpret_cast<const half8_t*>(sK + kLo + at), sh, ks[o][u]);
            }
          }
        }
      }
      const float so_down = xs_f[16 * (1 - r)];
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
            R[u][i] = fmaf(-f[i], fmaf(ks[1][u][i], so_down, ks[0][u][i] * s_down), v[4 * u + i]);
          }
        }
        sr = pow2_to_top(tiles_absmax<2>(R));
        tiles_to_operand<true>(R[0], R[1], sr.up, Rh, Rl);
        if (r == 0) {
          *piece(W::kXR, 0, 0) = Rh;
          *piece(W::kXR, 0, 1) = Rl;
          *xr_f = sr.down;
        }
      }
      __syncthreads();

      // E = T R
      f32x4_t E[2];
      {
        const float tri = sF[4 * kGdrC + 1], down = sr.down * tri;
        const auto T = [&](int f, int half) __attribute__((always_inline)) {
          return *reinterpret_cast<const half8_t*>(sT + (2 * f + half) * kGdrFragHalves + lane * 8);
        };
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int f = r == 0 ? u : 3 + 2 * u;
          const half8_t th = T(f, 0), tl = T(f, 1);
          f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          acc = mfma16(th, Rh, acc);
          acc = mfma16(th, Rl, acc);
          acc = mfma16(tl, Rh, acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) E[u][i] = acc[i] * down;
        }
        if (r == 1) {
          const half8_t oh = *piece(W::kXR, 0, 0), ol = *piece(W::kXR, 0, 1);
          const float other = *xr_f * tri;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const half8_t th = T(2 + 2 * u, 0), tl = T(2 + 2 * u, 1);
            f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            acc = mfma16(th, oh, acc);
            acc = mfma16(th, ol, acc);
            acc = mfma16(tl, oh, acc);
#pragma unroll
            for (int i = 0; i < 4; ++i) E[u][i] = fmaf(acc[i], other, E[u][i]);
          }
        }
      }
      // w E as an operand for both waves, E for the waves that form y.
      half8_t Dh, Dl;
      Pow2 sd;
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
        *piece(W::kXD, r, 0) = Dh;
        *piece(W::kXD, r, 1) = Dl;
        xd_f[16 * r] = sd.down;
        if constexpr (!KEEP) {
          half8_t Eh, El;
          const Pow2 se = pow2_to_top(tiles_absmax<2>(E));
          tiles_to_operand<true>(E[0], E[1], se.up, Eh, El);
          const int at = r == 0 ? W::kXE : W::kXR;
          *piece(at, 0, 0) = Eh;
          *piece(at, 0, 1) = El;
          xe_f[16 * r] = se.down;
        }
      }
      const float end = sF[4 * kGdrC];
      __syncthreads();

      // S' = e^(c_end) S + K^T (w E) on the wave's half of the rows
      {
        const half8_t oh = *piece(W::kXD, 1 - r, 0), ol = *piece(W::kXD, 1 - r, 1);
        const float d_own = sd.down, d_oth = xd_f[16 * (1 - r)];
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
          for (int i = 0; i < 4; ++i) S[j][i] = fmaf(acc[1][i], d_oth, fmaf(acc[0][i], d_own, end * S[j][i]));
        }
      }
      if (more) split_S();
      __syncthreads();
      if constexpr (W::NBUF == 1) __syncthreads();
      if constexpr (MODE == kGdrKeep) {
        const int64_t item = item0 + c;
        const rsrc_t re = raw_buffer(ws.E + item * kGdrC * P, static_cast<uint32_t>(kGdrC * P * 4));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t at = static_cast<uint32_t>((32 * r + 16 * (i / 4) + 4 * g + (i % 4)) * P + col) * 4;
          buffer_store_f32<false>(E[i / 4][i % 4], re, col_ok ? at : kOutOfRange);
        }
        buffer_store_f32<false>(lanes16_max(tiles_absmax<2>(E)), raw_buffer(ws.top + item * kGdrMaxima * kGdrMaxSlots, kGdrMaxima * kGdrMaxSlots * 4),
                                lane == 0 && col < P ? static_cast<uint32_t>(kMaxE * kGdrMaxSlots + col / 16 * 2 + r) * 4 : kOutOfRange);
      }
    }
    if (W::kLag && !lag) __syncthreads();
    if constexpr (MODE != kGdrKeep) {
      float* out = MODE == kGdrMap ? ws.map + (static_cast<int64_t>(walk_id) * cols + (col < cols ? col : 0)) * N
                                   : (p.h_final != nullptr && last_seg ? p.h_final + sb : nullptr);
      if (out != nullptr && col < cols) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = n0 + 32 * (j / 2) + 8 * g + 4 * (j & 1) + i;
            if (n < N) out[n] = S[j][i];
          }
        }
      }
    }
    return;
  }

  // ------------------------------------------------------- loads, and y
  const int ow = w - 2 * NPAIR, ltid = tid - 128 * NPAIR;
  const int pr = W::kHalvesOut == 2 ? ow : ow >> 1;
  const int col = col0 + 16 * pr + m;
  const bool col_ok = col < P;
  const _Float16* const xh = reinterpret_cast<const _Float16*>(xch[pr]);
  const float* const xf = reinterpret_cast<const float*>(xh + W::kXF);
  const float *const xs_f = xf + W::kSS + m, *const xe_f = xf + W::kSE + m;
  const auto piece = [&](int at, int q, int half) __attribute__((always_inline)) {
    return *reinterpret_cast<const half8_t*>(xh + at + (2 * q + half) * kGdrFragHalves + lane * 8);
  };
  u32x4_t kr[W::NKQ], qr[KEEP ? 1 : W::NKQ], tr[W::NTL], pm[KEEP ? 1 : W::NPL];
  float fr[W::NFL];
  f32x2_t fe;
  auto fetch_kq = [&](int c) __attribute__((always_inline)) {
    const float* fac = ws.fac + (item0 + c) * (kGdrFactors * kGdrC);
    const u32x4_t* K = reinterpret_cast<const u32x4_t*>(ws.K + (kv0 + c) * W::kMat) + ltid;
    const u32x4_t* Q = reinterpret_cast<const u32x4_t*>(ws.Q + (kv0 + c) * W::kMat) + ltid;
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      kr[i] = K[i * W::NL];
      if constexpr (!KEEP) qr[i] = Q[i * W::NL];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) fr[i] = fac[kFacK * kGdrC + (i * W::NL + ltid) % (4 * kGdrC)];
    fe = *reinterpret_cast<const f32x2_t*>(fac + kFacEnd * kGdrC);
  };
  auto fetch_T = [&](int c) __attribute__((always_inline)) {
    const u32x4_t* T = reinterpret_cast<const u32x4_t*>(ws.T + (item0 + c) * kGdrPieceHalves);
#pragma unroll
    for (int i = 0; i < W::NTL; ++i) tr[i] = T[(i * W::NL + ltid) % (W::kT / 8)];
  };
  auto fetch_P = [&](int c) __attribute__((always_inline)) {
    if constexpr (KEEP) return;
    const u32x4_t* Pm = reinterpret_cast<const u32x4_t*>(ws.Pm + (item0 + c) * kGdrPieceHalves);
#pragma unroll
    for (int i = 0; i < W::NPL; ++i) pm[i] = Pm[(i * W::NL + ltid) % (W::kP / 8)];  // (past the end: any)
  };
  // K, Q and the factors into a buffer.
  auto stage_kq = [&](int buf) __attribute__((always_inline)) {
    _Float16* sK = reinterpret_cast<_Float16*>(lds[buf]);
    float* sF = reinterpret_cast<float*>(sK + (KEEP ? 1 : 2) * W::kMat);
#pragma unroll
    for (int i = 0; i < W::NKQ; ++i) {
      reinterpret_cast<u32x4_t*>(sK)[i * W::NL + ltid] = kr[i];
      if constexpr (!KEEP) reinterpret_cast<u32x4_t*>(sK + W::kMat)[i * W::NL + ltid] = qr[i];
    }
#pragma unroll
    for (int i = 0; i < W::NFL; ++i) {
      const int e = i * W::NL + ltid;
      if (4 * kGdrC % W::NL == 0 || e < 4 * kGdrC) sF[e] = fr[i];
    }
    if (ltid == 0) *reinterpret_cast<f32x2_t*>(sF + 4 * kGdrC) = fe;
  };
  auto stage_T = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W::NTL; ++i) {
      const int e = i * W::NL + ltid;
      if (W::kT / 8 % W::NL == 0 || e < W::kT / 8) reinterpret_cast<u32x4_t*>(sT)[e] = tr[i];
    }
  };
  auto stage_P = [&]() __attribute__((always_inline)) {
    if constexpr (KEEP) return;
#pragma unroll
    for (int i = 0; i < W::NPL; ++i) {
      const int e = i * W::NL + ltid;
      if (W::kP / 8 % W::NL == 0 || e < W::kP / 8) reinterpret_cast<u32x4_t*>(sP)[e] = pm[i];
    }
  };
  // Byte offset of the wave's element (4 g, col) of a chunk of y; past any
  // buffer (and staying there with a chunk's rows added) where there is no column.
  constexpr uint32_t YB = OB16 ? 2 : 4;
  const uint32_t ybase = col_ok ? (static_cast<uint32_t>(4 * g) * yrow + static_cast<uint32_t>(col)) * YB : 0x80000000u;
  // Q S of a chunk, in its first phase.
  f32x4_t qs[KEEP ? 1 : W::kHalvesOut][2][2];
  auto readout = [&](int c) __attribute__((always_inline)) {
    const _Float16* sQ = reinterpret_cast<const _Float16*>(lds[W::NBUF == 2 ? (c & 1) : 0]) + W::kMat;
    const float* sF = reinterpret_cast<const float*>(sQ + W::kMat);
    if constexpr (!KEEP) {
#pragma unroll
      for (int hf = 0; hf < W::kHalvesOut; ++hf) {
        const int r = W::kHalvesOut == 2 ? hf : (ow & 1);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
#pragma unroll
          for (int u = 0; u < 2; ++u) qs[hf][o][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < NK; ++q) {
            const int f = o * NK + q;
            const half8_t sh = piece(W::kXS, f, 0), sl = piece(W::kXS, f, 1);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int at = kq_at<NP>(32 * r + 16 * u + m, 32 * f + 8 * g);
              const half8_t a = *reinterpret_cast<const half8_t*>(sQ + at);
              qs[hf][o][u] = mfma16(a, sh, qs[hf][o][u]);
              qs[hf][o][u] = mfma16(a, sl, qs[hf][o][u]);
              if constexpr (RAW == 2) {
                qs[hf][o][u] = mfma16(*reinterpret_cast<const half8_t*>(sQ + kLo + at), sh, qs[hf][o][u]);
              }
            }
          }
        }
        const float d0 = xs_f[0], d1 = xs_f[16];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4_t fq = *reinterpret_cast<const f32x4_t*>(sF + 1 * kGdrC + 32 * r + 16 * u + 4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qs[hf][0][u][i] = fq[i] * fmaf(qs[hf][1][u][i], d1, qs[hf][0][u][i] * d0);
          }
        }
      }
    }
  };
  // Its y, in its third.
  auto output = [&](int c) __attribute__((always_inline)) {
    const float* sF = reinterpret_cast<const float*>(reinterpret_cast<const _Float16*>(lds[W::NBUF == 2 ? (c & 1) : 0]) +
                                                     2 * W::kMat);
    if constexpr (!KEEP) {
      const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
      const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
      const int out_rows = static_cast<int>(L - t0 < kGdrC ? L - t0 : kGdrC);
      const rsrc_t ry = rows_buffer<OB16 ? 2 : 4>(p.y, (row_b + t0) * yrow + static_cast<int64_t>(h) * P, out_rows,
                                                  yrow, P);
      const auto Pm = [&](int f, int half) __attribute__((always_inline)) {
        return *reinterpret_cast<const half8_t*>(sP + (2 * f + half) * kGdrFragHalves + lane * 8);
      };
#pragma unroll
      for (int hf = 0; hf < W::kHalvesOut; ++hf) {
        const int r = W::kHalvesOut == 2 ? hf : (ow & 1);
        const int own = r == 0 ? W::kXE : W::kXR;
        const half8_t eh = piece(own, 0, 0), el = piece(own, 0, 1);
        const float e_own = xe_f[16 * r];
        f32x4_t pe[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int f = r == 0 ? u : 3 + 2 * u;
          f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          acc = mfma16(Pm(f, 0), eh, acc);
          acc = mfma16(Pm(f, 0), el, acc);
          acc = mfma16(Pm(f, 1), eh, acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) pe[u][i] = acc[i] * e_own;
        }
        if (r == 1) {
          const half8_t oh = piece(W::kXE, 0, 0), ol = piece(W::kXE, 0, 1);
          const float e_oth = xe_f[0];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            acc = mfma16(Pm(2 + 2 * u, 0), oh, acc);
            acc = mfma16(Pm(2 + 2 * u, 0), ol, acc);
            acc = mfma16(Pm(2 + 2 * u, 1), oh, acc);
#pragma unroll
            for (int i = 0; i < 4; ++i) pe[u][i] = fmaf(acc[i], e_oth, pe[u][i]);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4_t fp = *reinterpret_cast<const f32x4_t*>(sF + 3 * kGdrC + 32 * r + 16 * u + 4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) pe[u][i] = fmaf(fp[i], pe[u][i], qs[hf][0][u][i]);
        }
        if (rows < kGdrC) {  // steps behind the row's last: 0
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (32 * r + 16 * (i / 4) + 4 * g + (i % 4) >= rows) pe[i / 4][i % 4] = 0.0f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t t = static_cast<uint32_t>(32 * r + 16 * (i / 4) + (i % 4));
          buffer_store_f32<OB16>(pe[i / 4][i % 4], ry, ybase + t * yrow * YB);
        }
      }
    }
  };
  // A wave forms y in two phases of a chunk and moves data in the third. (A
  // fetch behind the last chunk fetches that again.)
  const bool lag = W::kLag && pr >= NPAIR / 2;
  const auto at_most = [&](int c) { return c < n_chunks ? c : n_chunks - 1; };
  const auto walk = [&](auto lags) __attribute__((always_inline)) {  // (a loop for either, its loads in no branch)
    constexpr bool LAG = decltype(lags)::value;
    if (n_chunks > 0) {
      fetch_kq(0);
      stage_kq(0);
      fetch_kq(at_most(1));
      fetch_T(0);
      fetch_P(0);
    }
    // As many stores behind these loads as y's are behind a later chunk's: the loads
    // are counted from the last access backwards, for the first chunk and the later
    // ones alike, and T would else be waited for with all of y's stores. (A buffer
    // of no bytes: nothing is written.)
    if constexpr (!LAG && !KEEP) {
      const rsrc_t none = raw_buffer(p.y, 0);
#pragma unroll
      for (int i = 0; i < 8 * W::kHalvesOut; ++i) buffer_store_f32<OB16>(0.0f, none, static_cast<uint32_t>(16 * i));
    }
    __syncthreads();
    for (int c = 0; c < n_chunks; ++c) {
      const auto move = [&]() __attribute__((always_inline)) {
        if constexpr (W::NBUF == 2) {
          stage_kq((c + 1) & 1);
          fetch_kq(at_most(c + 2));
        }
        fetch_T(at_most(c + 1));
        fetch_P(at_most(c + 1));
      };
      stage_T();
      if constexpr (!LAG) {
        readout(c);
      } else {
        if (c > 0) output(c - 1);
      }
      __syncthreads();
      stage_P();
      if constexpr (LAG) {
        readout(c);
      } else {
        move();
      }
      __syncthreads();
      if constexpr (LAG) {
        move();
      } else {
        output(c);
      }
      __syncthreads();
      if constexpr (W::NBUF == 1) {
        stage_kq(0);
        fetch_kq(at_most(c + 2));
        __syncthreads();
      }
    }
    if constexpr (LAG) {
      if (n_chunks > 0) output(n_chunks - 1);
    }
    if constexpr (W::kLag) __syncthreads();
  };
  if constexpr (W::kLag) {
    if (lag) {
      walk(std::true_type{});
    } else {
      walk(std::false_type{});
    }
  } else {
    walk(std::false_type{});
  }

  if constexpr (KEEP) return;
  // Steps behind the row's last: zeros from the first chunk that was not walked.
  constexpr int kPart = W::kHalvesOut == 2 ? 1 : 2;
  for (int64_t t = static_cast<int64_t>(n_chunks) * kGdrC + 4 * (ow % kPart) + g; t < L; t += 4 * kPart) {
    if (col_ok) store_elem<OB16>(p.y, (row_b + t) * yrow + static_cast<int64_t>(h) * P + col, 0.0f);
  }
}

template <int NP, bool BF16, bool OB16, int NPAIR, int MODE>
__global__ __launch_bounds__((GdrWalk<NP, BF16, OB16, NPAIR, MODE>::NT)) void gdr_chunk_kernel(const GatedDeltaArgs p,
                                                                                             const GdrWork ws,
                                                                                             int chunks, int segs,
                                                                                             int seg_chunks) {
  __shared__ GdrWalkLds<GdrWalk<NP, BF16, OB16, NPAIR, MODE>, NPAIR> lds;
  gdr_walk<NP, BF16, OB16, NPAIR, MODE>(p, ws, chunks, segs, seg_chunks, static_cast<int>(blockIdx.x),
                                        static_cast<int>(threadIdx.x), lds);
}

template <int NP, bool BF16, bool OB16, int MODE>
void gdr_launch_chunk_pairs(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, int segs, int seg_chunks,
                            hipStream_t st) {
  const int64_t walks = a.batch * a.nheads * segs;
  const int64_t slices = (a.headdim + (MODE == kGdrMap ? a.dstate : 0) + 15) / 16;
  const int pairs = gdr_block_pairs(walks, slices);
  const auto blocks = [&](int n) { return static_cast<unsigned>(walks * ((slices + n - 1) / n)); };
  using W4 = GdrWalk<NP, BF16, OB16, 4, MODE>;
  if constexpr (W4::kFits) {
    if (pairs == 4) {
      gdr_chunk_kernel<NP, BF16, OB16, 4, MODE><<<blocks(4), W4::NT, 0, st>>>(a, ws, chunks, segs, seg_chunks);
      return;
    }
  }
  if (pairs == 1) {
    if constexpr (MODE != kGdrKeep || !gdr_both_fit(NP, BF16)) {
      gdr_chunk_kernel<NP, BF16, OB16, 1, MODE>
          <<<blocks(1), GdrWalk<NP, BF16, OB16, 1, MODE>::NT, 0, st>>>(a, ws, chunks, segs, seg_chunks);
    }
  } else {
    gdr_chunk_kernel<NP, BF16, OB16, 2, MODE>
        <<<blocks(2), GdrWalk<NP, BF16, OB16, 2, MODE>::NT, 0, st>>>(a, ws, chunks, segs, seg_chunks);
  }
}

template <bool BF16>
int gdr_launch_chunk(const GatedDeltaArgs& a, const GdrWork& ws, const GdrPlan& pl, bool backward, hipStream_t st) {
  const int chunks = static_cast<int>(pl.chunks), segs = static_cast<int>(pl.segs);
  const int seg_chunks = static_cast<int>(pl.seg_chunks);
  const auto types = [&](auto np) {
    constexpr int NP = decltype(np)::value;
    if (backward) {
      gdr_launch_chunk_pairs<NP, BF16, true, kGdrKeep>(a, ws, chunks, 1, chunks, st);
      return;
    }
    if (segs > 1) {
      gdr_launch_chunk_pairs<NP, BF16, true, kGdrMap>(a, ws, chunks, segs, seg_chunks, st);
      launch_gdr_join(a, ws, segs, seg_chunks, st);
    }
    if (a.out_bf16) {
      gdr_launch_chunk_pairs<NP, BF16, true, kGdrForward>(a, ws, chunks, segs, seg_chunks, st);
    } else {
      gdr_launch_chunk_pairs<NP, BF16, false, kGdrForward>(a, ws, chunks, segs, seg_chunks, st);
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
