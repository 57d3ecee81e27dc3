// Gated delta rule, the part of a chunk that does not depend on the state: the
// halves of K and Q, the triangular inverse T, the output's weights Pm and the per-step factors, for
// every chunk at once.
//
// One block of four waves per (batch row, query/key head, chunk); the value
// heads that share q and k are taken one after another. K K^T and Q K^T (the
// ten lower 16 x 16 tiles each) run on the matrix cores and stay in registers.
// M = L diag(beta) is strictly lower, and T = (1 + M)^-1 is found by
// substitution, never by powers of M (with equal keys and no decay the powers
// reach 10^18 and cancel): one wave inverts the four diagonal blocks, a column
// a lane, while the others write out Pm; then wave w takes block column w of T
// down the rows, T_iw = -T_ii sum_k M_ik T_kw, in float32 matrix instructions,
// without leaving its registers.
// Sums of log decays and their differences are in double: behind a step that
// forgets nearly everything the sums are large and the differences small.
#include <hip/hip_runtime.h>

#include "gdr_mma.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kMS = kGdrC + 4;  // row stride of the float32 matrices in LDS

__device__ __forceinline__ f32x4_t mfma4(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// acc += A X for 16 x 16 tiles: A from LDS (row-major), X a D tile. Step s of
// the four contracts rows 4 g + s, which is where X's element s lives.
__device__ __forceinline__ f32x4_t tile_product(const float* A, f32x4_t X, f32x4_t acc, int m, int g) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(A + m * kMS + 4 * g);
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = mfma4(a[s], X[s], acc);
  return acc;
}

// BWD: also the pieces of T^T and, in place of Pm's, those of Pm^T.
template <int NP, bool BF16, bool VEC, bool BWD>
__global__ __launch_bounds__(kThreads) void gdr_prep_kernel(const GatedDeltaArgs p, const GdrWork ws, int chunks,
                                                            int out_lo) {
  constexpr int RAW = BF16 ? 1 : 2;
  constexpr int kMat = RAW * kGdrC * NP;              // halves of K (or Q)
  constexpr int kKQ = 2 * kMat * 2;                   // bytes
  constexpr int kTP = 2 * kGdrC * kMS * 4;
  __shared__ __align__(16) char pool[kKQ > kTP ? kKQ : kTP];  // K and Q, then T and Pm
  __shared__ __align__(16) float sM[kGdrC * kMS];
  __shared__ double sC[kGdrC];
  __shared__ float sTop[4];
  __shared__ __align__(16) float sBeta[kGdrC], sKn[kGdrC], sQn[kGdrC], sKup[kGdrC], sQup[kGdrC];
  _Float16* sK = reinterpret_cast<_Float16*>(pool);   // [RAW][64][NP]
  _Float16* sQ = sK + kMat;
  float* sT = reinterpret_cast<float*>(pool);         // [64][kMS]
  float* sP = sT + kGdrC * kMS;

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads), heads = H / G;
  const int c = static_cast<int>(blockIdx.x) % chunks;
  const int bg = static_cast<int>(blockIdx.x) / chunks;
  const int b = bg / G, kh = bg % G;
  const int64_t len = gdr_row_steps(p.seqlens, b, p.seqlen);
  const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
  if (t0 >= len) return;  // behind the row's last step: nothing reads this chunk
  const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
  const int64_t row0 = static_cast<int64_t>(b) * p.seqlen + t0;

  gdr_stage_kq<NP, BF16, VEC>(p, row0, rows, kh, tid, sK, sQ, ws.K + static_cast<int64_t>(blockIdx.x) * kMat,
                              ws.Q + static_cast<int64_t>(blockIdx.x) * kMat, sKn, sQn, sKup, sQup);
  __syncthreads();

  // The ten lower tiles of K K^T and Q K^T, q = w, w + 4, w + 8, times the
  // rows' factors.
  f32x4_t kk[3], qk[3];
  const auto tile = [&](int j, int& ti, int& si) __attribute__((always_inline)) {
    const int q = w + 4 * j;
    ti = q == 0 ? 0 : (q < 3 ? 1 : (q < 6 ? 2 : 3));
    si = q - ti * (ti + 1) / 2;
    return q < 10;
  };
  {
  const int m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    int ti, si;
    kk[j] = qk[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (!tile(j, ti, si)) continue;
#pragma unroll
    for (int n = 0; n < NP; n += 32) {
      const int at = kq_at<NP>(16 * ti + m, n + 8 * g), bt = kq_at<NP>(16 * si + m, n + 8 * g);
      const half8_t bk = *reinterpret_cast<const half8_t*>(sK + bt);
      const half8_t ak = *reinterpret_cast<const half8_t*>(sK + at);
      const half8_t aq = *reinterpret_cast<const half8_t*>(sQ + at);
      kk[j] = mfma16(ak, bk, kk[j]);
      qk[j] = mfma16(aq, bk, qk[j]);
      if constexpr (RAW == 2) {
        const half8_t bl = *reinterpret_cast<const half8_t*>(sK + kGdrC * NP + bt);
        kk[j] = mfma16(ak, bl, kk[j]);
        qk[j] = mfma16(aq, bl, qk[j]);
        kk[j] = mfma16(*reinterpret_cast<const half8_t*>(sK + kGdrC * NP + at), bk, kk[j]);
        qk[j] = mfma16(*reinterpret_cast<const half8_t*>(sQ + kGdrC * NP + at), bk, qk[j]);
      }
    }
    const f32x4_t kt = *reinterpret_cast<const f32x4_t*>(sKn + 16 * ti + 4 * g);
    const f32x4_t qt = *reinterpret_cast<const f32x4_t*>(sQn + 16 * ti + 4 * g);
    const float ks = sKn[16 * si + m];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kk[j][i] *= kt[i] * ks;
      qk[j][i] *= qt[i] * (ks * p.scale);
    }
  }
  }

  for (int hh = 0; hh < heads; ++hh) {
    const int place = anew(lane), m = place & 15, g = place >> 4;
    const int h = kh * heads + hh;
    const int64_t item = (static_cast<int64_t>(b) * H + h) * chunks + c;
    // Gates: lane t of wave 0. (Sums in units of log 2, for the base-2 exponential.)
    if (w == 0) {
      float ld = 0.0f, beta = 0.0f;
      if (lane < rows) {
        const int64_t at = (row0 + lane) * H + h;
        ld = gdr_log_decay(p, load_elem<BF16>(p.dt, at), p.dt_bias ? p.dt_bias[h] : 0.0f, p.A[h]);
        beta = gdr_beta(p, load_elem<BF16>(p.beta, at));
      }
      sC[lane] = wave_prefix(static_cast<double>(ld) * kLog2eD, lane);
      sBeta[lane] = beta;
    }
    __syncthreads();  // gates; K and Q (or the last head's T and Pm) are done with

#pragma unroll
    for (int j = 0; j < 3; ++j) {
      int ti, si;
      if (!tile(j, ti, si)) continue;
      const int s = 16 * si + m;
      const double cs = sC[s];
      const float bs = sBeta[s];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * ti + 4 * g + i;
        const float dec = exp2_hw(static_cast<float>(sC[t] - cs)) * bs;
        sM[t * kMS + s] = t > s ? dec * kk[j][i] : 0.0f;
        sP[t * kMS + s] = t >= s ? dec * qk[j][i] : 0.0f;
      }
    }
    __syncthreads();

    float* fac = ws.fac + item * (kGdrFactors * kGdrC);
    // Row tile `tt` of a matrix (or of its transpose) as halves in the order a
    // lane feeds them, scaled by rows, or by a given power of two.
    const auto pieces = [&](const float* src, int tt, bool up, _Float16* out, float* down, bool lo, bool whole,
                            Pow2 given) __attribute__((always_inline)) {
      const int place = anew(lane), m = place & 15, g = place >> 4;
      const int t = 16 * tt + m;
      float x[2][8];
      float top = 0.0f;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (up ? (q == 0 && tt >= 2) : (q == 1 && tt < 2)) continue;
        if (!up) {
          const f32x4_t a = *reinterpret_cast<const f32x4_t*>(src + t * kMS + 32 * q + 4 * g);
          const f32x4_t d = *reinterpret_cast<const f32x4_t*>(src + t * kMS + 32 * q + 16 + 4 * g);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[q][e] = a[e], x[q][4 + e] = d[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int s = 32 * q + (e < 4 ? 4 * g + e : 12 + 4 * g + e);
          // (a block above the diagonal was never written)
          if (up) x[q][e] = src[s * kMS + t];
          if (up ? s < t : s > t) x[q][e] = 0.0f;
          top = fmaxf(top, fabsf(x[q][e]));
        }
      }
      const Pow2 s = whole ? given : pow2_to_top(col_max(top));
      if (!whole && g == 0) down[t] = s.down;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (up ? (q == 0 && tt >= 2) : (q == 1 && tt < 2)) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[q][e] *= s.up;
        const half8_t hi = halves(x[q]);
        _Float16* at = out + (up ? gdr_frag_up(tt, q) : gdr_frag(tt, q)) * 2 * kGdrFragHalves + lane * 8;
        *reinterpret_cast<half8_t*>(at) = hi;
        if (lo) *reinterpret_cast<half8_t*>(at + kGdrFragHalves) = rest(x[q], hi);
      }
    };

    // Wave 0: the diagonal blocks' inverses, lane (g, m) column m of block g.
    // The others: Pm, and the factors.
    if (w == 0) {
      float x[16];
      const float* D = sM + 16 * g * kMS + 16 * g;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float acc = i == m ? 1.0f : 0.0f;
#pragma unroll
        for (int k = 0; k < i; ++k) acc = fmaf(-D[i * kMS + k], x[k], acc);
        x[i] = acc;
        sT[(16 * g + i) * kMS + 16 * g + m] = acc;
      }
    } else {
      const Pow2 none = Pow2{1.0f, 1.0f};
      _Float16* out = (BWD ? ws.Pt : ws.Pm) + item * kGdrPieceHalves;
      pieces(sP, w, BWD, out, fac + kFacP * kGdrC, BWD || out_lo, false, none);
      if (w == 1) pieces(sP, 0, BWD, out, fac + kFacP * kGdrC, BWD || out_lo, false, none);
      if (w == 2) {
        const double ct = sC[lane], cend = sC[kGdrC - 1];
        const float into = exp2_hw(static_cast<float>(ct));
        const float last = exp2_hw(static_cast<float>(cend - ct));
        fac[kFacK * kGdrC + lane] = into * sKn[lane];
        fac[kFacQ * kGdrC + lane] = p.scale * into * sQn[lane];
        fac[kFacW * kGdrC + lane] = sBeta[lane] * last * sKn[lane];
        if constexpr (BWD) {
          fac[kFacKup * kGdrC + lane] = sKup[lane];
          fac[kFacQup * kGdrC + lane] = sQup[lane];
          fac[kFacKn * kGdrC + lane] = sKn[lane];
          fac[kFacQn * kGdrC + lane] = sQn[lane];
        }
        if (lane == 0) fac[kFacEnd * kGdrC] = exp2_hw(static_cast<float>(cend));
      }
    }
    __syncthreads();

    // Block column w of T.
    float top = 0.0f;
    {
      f32x4_t T[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        T[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (i == w) {
#pragma unroll
          for (int e = 0; e < 4; ++e) T[i][e] = sT[(16 * i + 4 * g + e) * kMS + 16 * i + m];
        }
        if (i > w) {
          f32x4_t X = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < i; ++k) {
            if (k >= w) X = tile_product(sM + 16 * i * kMS + 16 * k, T[k], X, m, g);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) X[e] = -X[e];
          T[i] = tile_product(sT + 16 * i * kMS + 16 * i, X, T[i], m, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) sT[(16 * i + 4 * g + e) * kMS + 16 * w + m] = T[i][e];
        }
      }
      top = lanes16_max(tiles_absmax<4>(T));
    }
    if (lane == 0) sTop[w] = top;
    __syncthreads();

    // T by one power of two for the whole triangle: its rows all have a 1, and
    // halves reach down to 2^-38 of the largest element.
    const Pow2 st = pow2_to_top(fmaxf(fmaxf(sTop[0], sTop[1]), fmaxf(sTop[2], sTop[3])));
    if (tid == 0) fac[kFacEnd * kGdrC + 1] = st.down;
    pieces(sT, w, false, ws.T + item * kGdrPieceHalves, nullptr, true, true, st);
    if constexpr (BWD) pieces(sT, w, true, ws.Tt + item * kGdrPieceHalves, nullptr, true, true, st);
  }
}

template <int NP, bool BF16, bool VEC>
void launch_np(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, unsigned blocks, int out_lo, bool backward,
               hipStream_t st) {
  if (backward) {
    gdr_prep_kernel<NP, BF16, VEC, true><<<blocks, kThreads, 0, st>>>(a, ws, chunks, out_lo);
  } else {
    gdr_prep_kernel<NP, BF16, VEC, false><<<blocks, kThreads, 0, st>>>(a, ws, chunks, out_lo);
  }
}

template <int NP, bool BF16>
void launch_vec(const GatedDeltaArgs& a, const GdrWork& ws, int chunks, unsigned blocks, int out_lo, bool backward,
                bool vec, hipStream_t st) {
  vec ? launch_np<NP, BF16, true>(a, ws, chunks, blocks, out_lo, backward, st)
      : launch_np<NP, BF16, false>(a, ws, chunks, blocks, out_lo, backward, st);
}

}  // namespace

int launch_gdr_prep(const GatedDeltaArgs& a, const GdrWork& ws, int64_t chunks, int out_lo, bool backward, bool vec,
                    void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const unsigned blocks = static_cast<unsigned>(a.batch * a.nkheads * chunks);
  const int n = static_cast<int>(chunks);
  if (a.dstate <= 64) {
    a.in_bf16 ? launch_vec<64, true>(a, ws, n, blocks, out_lo, backward, vec, st)
              : launch_vec<64, false>(a, ws, n, blocks, out_lo, backward, vec, st);
  } else {
    a.in_bf16 ? launch_vec<128, true>(a, ws, n, blocks, out_lo, backward, vec, st)
              : launch_vec<128, false>(a, ws, n, blocks, out_lo, backward, vec, st);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
