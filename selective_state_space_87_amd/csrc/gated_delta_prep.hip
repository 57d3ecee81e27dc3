// Gated delta rule, the part of a chunk that does not depend on the state: the
// halves of K and Q, the triangular inverse T, the output's weights Pm and the
// per-step factors, for every chunk at once.
//
// One block of four waves per (batch row, query/key head, chunk); the value
// heads that share q and k are taken one after another, or, where that leaves
// compute units without a block, by a block each. K K^T and K Q^T (the
// ten 16 x 16 tiles of a triangle each) run on the matrix cores and stay in
// registers: K Q^T, not Q K^T, since the D of its tiles is then, two tiles
// together, the operand that Pm is fed as (lane m has row m of Pm, its elements
// are 4 consecutive columns of either tile), with no way through LDS.
// M = L diag(beta) is strictly lower, and T = (1 + M)^-1 is found by
// substitution, never by powers of M (with equal keys and no decay the powers
// reach 10^18 and cancel): one wave inverts the four diagonal blocks, a column
// a lane; then wave w takes block row w of T leftwards,
//   T_wj = -(sum_(k > j) T_wk M_kj) T_jj,
// transposed, in float32 matrix instructions, without leaving its registers,
// and has again in D what T is fed as. (The backward's T^T: the same by block columns.)
// Sums of log decays are in double, and kept as two floats whose differences
// are taken apart: behind a step that forgets nearly everything the sums are
// large and the differences small.
// Measured at (4, 8192, 16 key and 32 value heads of 128 x 128), bfloat16: 191 us
// for 0.28 GB in and 0.69 GB out, 5.1 TB/s. (T through LDS and stored from there 22 us more.)
#include <hip/hip_runtime.h>

#include "gdr_mma.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kMS = kGdrC + 4;  // row stride of M in LDS (floats)
constexpr int kDS = 16 + 4;     // row stride of a diagonal block's inverse

__device__ __forceinline__ f32x4_t mfma4(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// acc += A X for 16 x 16 tiles: A from LDS (row-major, or TR its transpose), X
// a D tile. Step s of the four contracts rows 4 g + s, which is where X's element s lives.
template <bool TR>
__device__ __forceinline__ f32x4_t tile_product(const float* A, int stride, f32x4_t X, f32x4_t acc, int m, int g) {
  f32x4_t a;
  if constexpr (TR) {
#pragma unroll
    for (int s = 0; s < 4; ++s) a[s] = A[(4 * g + s) * stride + m];
  } else {
    a = *reinterpret_cast<const f32x4_t*>(A + m * stride + 4 * g);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = mfma4(a[s], X[s], acc);
  return acc;
}

// The two D tiles 2 q, 2 q + 1 as a piece: its halves times `up`.
__device__ __forceinline__ void store_piece(_Float16* at, f32x4_t a, f32x4_t b, float up) {
  const float x[8] = {a[0] * up, a[1] * up, a[2] * up, a[3] * up, b[0] * up, b[1] * up, b[2] * up, b[3] * up};
  const half8_t hi = halves(x);
  *reinterpret_cast<half8_t*>(at) = hi;
  *reinterpret_cast<half8_t*>(at + kGdrFragHalves) = rest(x, hi);
}

// BWD: also the pieces of T^T and, in place of Pm's, those of Pm^T.
template <int NP, bool BF16, bool VEC, bool BWD>
__global__ __launch_bounds__(kThreads) void gdr_prep_kernel(const GatedDeltaArgs p, const GdrWork ws, int chunks,
                                                            int blocks_a_group) {
  constexpr int RAW = BF16 ? 1 : 2;
  constexpr int kMat = RAW * kGdrC * NP;              // halves of K (or Q)
  constexpr int kKQ = 2 * kMat * 2;                   // bytes
  constexpr int kMD = (kGdrC * kMS + 4 * 16 * kDS) * 4;
  __shared__ __align__(16) char pool[kKQ > kMD ? kKQ : kMD];  // K and Q, then M and the diagonal inverses
  __shared__ float sCh[kGdrC], sCl[kGdrC];            // sums of log decays in units of log 2, hi + lo
  __shared__ float sTop[4];
  __shared__ __align__(16) float sBeta[kGdrC], sKn[kGdrC], sQn[kGdrC], sKup[kGdrC], sQup[kGdrC];
  _Float16* sK = reinterpret_cast<_Float16*>(pool);   // [RAW][64][NP]
  _Float16* sQ = sK + kMat;
  float* sM = reinterpret_cast<float*>(pool);         // [64][kMS]
  float* sD = sM + kGdrC * kMS;                       // [4][16][kDS]

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads), heads = H / G;
  const int group = static_cast<int>(blockIdx.x) / blocks_a_group;  // (batch row, query/key head, chunk)
  const int first = static_cast<int>(blockIdx.x) % blocks_a_group;  // the block's heads: one, or all
  const int behind = blocks_a_group > 1 ? first + 1 : heads;
  const int c = group % chunks;
  const int bg = group / chunks;
  const int b = bg / G, kh = bg % G;
  const int64_t len = gdr_row_steps(p.seqlens, b, p.seqlen);
  const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
  if (t0 >= len) return;  // behind the row's last step: nothing reads this chunk
  const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
  const int64_t row0 = static_cast<int64_t>(b) * p.seqlen + t0;

  // The gates of a head, read before the work in front of their use (lane t has
  // step t; loads in no branch).
  const int64_t gate_row = (row0 + (lane < rows ? lane : rows - 1)) * H + kh * heads;
  float dt_raw, beta_raw, dt_bias, A;
  const auto fetch_gates = [&](int hh) __attribute__((always_inline)) {
    dt_raw = load_elem<BF16>(p.dt, gate_row + hh);
    beta_raw = load_elem<BF16>(p.beta, gate_row + hh);
    dt_bias = p.dt_bias ? p.dt_bias[kh * heads + hh] : 0.0f;
    A = p.A[kh * heads + hh];
  };
  fetch_gates(first);

  gdr_stage_kq<NP, BF16, VEC>(p, row0, rows, kh, tid, sK, sQ, first == 0,
                              ws.K + static_cast<int64_t>(group) * kMat, ws.Q + static_cast<int64_t>(group) * kMat, sKn, sQn, sKup, sQup);
  __syncthreads();

  // K K^T: the ten lower tiles, tile q = w, w + 4, w + 8. For Pm: K Q^T, its
  // tiles (s-tile j, t-tile w), j <= w (D: lane m step t, elements steps s);
  // for Pm^T: Q K^T, tiles (t-tile j, s-tile w), j >= w. Times the rows' factors.
  f32x4_t kk[3], pq[4];
  const auto tile = [&](int j, int& ti, int& si) __attribute__((always_inline)) {
    const int q = w + 4 * j;
    ti = q == 0 ? 0 : (q < 3 ? 1 : (q < 6 ? 2 : 3));
    si = q - ti * (ti + 1) / 2;
    return q < 10;
  };
  const auto in_row = [&](int j) __attribute__((always_inline)) { return BWD ? j >= w : j <= w; };
  {
    const int m = lane & 15, g = lane >> 4;
    // A B^T for 16-row tiles of two matrices of halves.
    const auto product = [&](const _Float16* A, int ta, const _Float16* B, int tb) __attribute__((always_inline)) {
      f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < NP; n += 32) {
        const int at = kq_at<NP>(16 * ta + m, n + 8 * g), bt = kq_at<NP>(16 * tb + m, n + 8 * g);
        const half8_t x = *reinterpret_cast<const half8_t*>(A + at), y = *reinterpret_cast<const half8_t*>(B + bt);
        acc = mfma16(x, y, acc);
        if constexpr (RAW == 2) {
          acc = mfma16(x, *reinterpret_cast<const half8_t*>(B + kGdrC * NP + bt), acc);
          acc = mfma16(*reinterpret_cast<const half8_t*>(A + kGdrC * NP + at), y, acc);
        }
      }
      return acc;
    };
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      int ti, si;
      kk[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (!tile(j, ti, si)) continue;
      kk[j] = product(sK, ti, sK, si);
      const f32x4_t kt = *reinterpret_cast<const f32x4_t*>(sKn + 16 * ti + 4 * g);
      const float ks = sKn[16 * si + m];
#pragma unroll
      for (int i = 0; i < 4; ++i) kk[j][i] *= kt[i] * ks;
    }
    const float own = (BWD ? sKn : sQn)[16 * w + m] * p.scale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      pq[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (!in_row(j)) continue;
      pq[j] = product(BWD ? sQ : sK, j, BWD ? sK : sQ, w);
      const f32x4_t f = *reinterpret_cast<const f32x4_t*>((BWD ? sQn : sKn) + 16 * j + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) pq[j][i] *= f[i] * own;
    }
  }

  for (int hh = first; hh < behind; ++hh) {
    const int place = anew(lane), m = place & 15, g = place >> 4;
    const int h = kh * heads + hh;
    const int64_t item = (static_cast<int64_t>(b) * H + h) * chunks + c;
    float* fac = ws.fac + item * (kGdrFactors * kGdrC);
    // Gates: lane t of wave 0. (Sums in units of log 2, for the base-2 exponential.)
    if (w == 0) {
      const float ld = lane < rows ? gdr_log_decay(p, dt_raw, dt_bias, A) : 0.0f;
      const double cs = wave_prefix(static_cast<double>(ld) * kLog2eD, lane);
      sCh[lane] = static_cast<float>(cs);
      sCl[lane] = static_cast<float>(cs - static_cast<double>(static_cast<float>(cs)));
      sBeta[lane] = lane < rows ? gdr_beta(p, beta_raw) : 0.0f;
    }
    fetch_gates(hh + 1 < behind ? hh + 1 : hh);
    __syncthreads();  // gates; K and Q (or the last head's M) are done with
    const auto decay = [&](float hi, float lo, float hi0, float lo0) __attribute__((always_inline)) {
      return exp2_hw((hi - hi0) + (lo - lo0));
    };

#pragma unroll
    for (int j = 0; j < 3; ++j) {
      int ti, si;
      if (!tile(j, ti, si)) continue;
      const int s = 16 * si + m;
      const float hs = sCh[s], ls = sCl[s], bs = sBeta[s];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * ti + 4 * g + i;
        const float v = decay(sCh[t], sCl[t], hs, ls) * (bs * kk[j][i]);
        sM[t * kMS + s] = ti != si || t > s ? v : 0.0f;
      }
    }
    __syncthreads();

    // Wave 0: the diagonal blocks' inverses, lane (g, m) column m of block g.
    if (w == 0) {
      float x[16];
      const float* D = sM + 16 * g * kMS + 16 * g;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float acc = i == m ? 1.0f : 0.0f;
#pragma unroll
        for (int k = 0; k < i; ++k) acc = fmaf(-D[i * kMS + k], x[k], acc);
        x[i] = acc;
        sD[(16 * g + i) * kDS + m] = acc;
      }
    }
    // Row tile w of Pm (or of Pm^T), scaled by rows.
    {
      f32x4_t x[4];
      float top = 0.0f;
      const int own = 16 * w + m;
      const float ho = sCh[own], lo = sCl[own], bo = BWD ? sBeta[own] : 1.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (!in_row(j)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int o = 16 * j + 4 * g + i;  // s (or t)
          const float d = BWD ? decay(sCh[o], sCl[o], ho, lo) * bo : decay(ho, lo, sCh[o], sCl[o]) * sBeta[o];
          const float v = d * pq[j][i];
          x[j][i] = j != w || (BWD ? o >= own : o <= own) ? v : 0.0f;
          top = fmaxf(top, fabsf(x[j][i]));
        }
      }
      const Pow2 s = pow2_to_top(col_max(top));
      if (g == 0) fac[kFacP * kGdrC + own] = s.down;
      _Float16* out = (BWD ? ws.Pt : ws.Pm) + item * kGdrPieceHalves + lane * 8;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (BWD ? (q == 0 && w >= 2) : (q == 1 && w < 2)) continue;
        store_piece(out + (BWD ? gdr_frag_up(w, q) : gdr_frag(w, q)) * 2 * kGdrFragHalves, x[2 * q], x[2 * q + 1], s.up);
      }
    }
    if (w == 1) {
      const float ht = sCh[lane], lt = sCl[lane];
      const float into = exp2_hw(ht + lt);
      const float last = decay(sCh[kGdrC - 1], sCl[kGdrC - 1], ht, lt);
      fac[kFacK * kGdrC + lane] = into * sKn[lane];
      fac[kFacQ * kGdrC + lane] = p.scale * into * sQn[lane];
      fac[kFacW * kGdrC + lane] = sBeta[lane] * last * sKn[lane];
      if constexpr (BWD) {
        fac[kFacKup * kGdrC + lane] = sKup[lane];
        fac[kFacQup * kGdrC + lane] = sQup[lane];
        fac[kFacKn * kGdrC + lane] = sKn[lane];
        fac[kFacQn * kGdrC + lane] = sQn[lane];
      }
      if (lane == kGdrC - 1) fac[kFacEnd * kGdrC] = into;
    }
    __syncthreads();

    // Block row w of T, transposed: R[j] is T_wj^T (lane m row t of T, elements
    // its columns s). R_j = -T_jj^T sum_(k > j) M_kj^T R_k.
    f32x4_t R[4], C[4];
    float top = 0.0f;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
      R[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (j == w) {
        R[j] = *reinterpret_cast<const f32x4_t*>(sD + (16 * j + m) * kDS + 4 * g);  // (T_jj^T)[4 g + i][m]
      }
      if (j < w) {
        f32x4_t X = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 3; k > j; --k) {
          if (k <= w) X = tile_product<true>(sM + 16 * k * kMS + 16 * j, kMS, R[k], X, m, g);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) X[e] = -X[e];
        R[j] = tile_product<true>(sD + 16 * j * kDS, kDS, X, R[j], m, g);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(R[j][e]));
    }
    if constexpr (BWD) {  // block column w: C[i] = T_iw
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        C[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (i == w) {
#pragma unroll
          for (int e = 0; e < 4; ++e) C[i][e] = sD[(16 * i + 4 * g + e) * kDS + m];
        }
        if (i > w) {
          f32x4_t X = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < i; ++k) {
            if (k >= w) X = tile_product<false>(sM + 16 * i * kMS + 16 * k, kMS, C[k], X, m, g);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) X[e] = -X[e];
          C[i] = tile_product<false>(sD + 16 * i * kDS, kDS, X, C[i], m, g);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(C[i][e]));
      }
    }
    top = lanes16_max(col_max(top));
    if (lane == 0) sTop[w] = top;
    __syncthreads();

    // T by one power of two for the whole triangle: its rows all have a 1, and
    // halves reach down to 2^-38 of the largest element.
    const Pow2 st = pow2_to_top(fmaxf(fmaxf(sTop[0], sTop[1]), fmaxf(sTop[2], sTop[3])));
    if (tid == 0) fac[kFacEnd * kGdrC + 1] = st.down;
    _Float16* out = ws.T + item * kGdrPieceHalves + lane * 8;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (q == 1 && w < 2) continue;
      store_piece(out + gdr_frag(w, q) * 2 * kGdrFragHalves, R[2 * q], R[2 * q + 1], st.up);
    }
    if constexpr (BWD) {
      out = ws.Tt + item * kGdrPieceHalves + lane * 8;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (q == 0 && w >= 2) continue;
        store_piece(out + gdr_frag_up(w, q) * 2 * kGdrFragHalves, C[2 * q], C[2 * q + 1], st.up);
      }
    }
  }
}

template <int NP, bool BF16, bool VEC>
void launch_np(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, unsigned blocks, int a_group,
               bool backward, hipStream_t st) {
  if (backward) {
    gdr_prep_kernel<NP, BF16, VEC, true><<<blocks, kThreads, 0, st>>>(a, ws, chunks, a_group);
  } else {
    gdr_prep_kernel<NP, BF16, VEC, false><<<blocks, kThreads, 0, st>>>(a, ws, chunks, a_group);
  }
}

template <int NP, bool BF16>
void launch_vec(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, unsigned blocks, int a_group,
                bool backward, bool vec, hipStream_t st) {
  vec ? launch_np<NP, BF16, true>(a, ws, chunks, blocks, a_group, backward, st)
      : launch_np<NP, BF16, false>(a, ws, chunks, blocks, a_group, backward, st);
}

}  // namespace

int launch_gdr_prep(const GatedDeltaArgs& a, const GdrWork& ws, int64_t chunks, bool backward, bool vec,
                    void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  // Measured (a whole forward, a block a group against a block a head): 2 groups
  // of 2 heads 21.8 us, 17.9; 4 of 4 heads 30.5, 19.0; 78 of 2 47.1, 43.3; 256 of 4
  // 134, 128; 512 of 2 61.5, 61.8; 1024 of 4 277, 290.
  constexpr int64_t kGroupsEnough = 512;
  const int64_t groups = a.batch * a.nkheads * chunks;
  const int a_group = groups < kGroupsEnough ? static_cast<int>(a.nheads / a.nkheads) : 1;
  const unsigned blocks = static_cast<unsigned>(groups * a_group);
  const int n = static_cast<int>(chunks);
  if (a.dstate <= 64) {
    a.in_bf16 ? launch_vec<64, true>(a, ws, n, blocks, a_group, backward, vec, st)
              : launch_vec<64, false>(a, ws, n, blocks, a_group, backward, vec, st);
  } else {
    a.in_bf16 ? launch_vec<128, true>(a, ws, n, blocks, a_group, backward, vec, st)
              : launch_vec<128, false>(a, ws, n, blocks, a_group, backward, vec, st);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
