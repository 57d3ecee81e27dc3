// Gated delta rule, the part of a chunk that does not depend on the state: the
// triangular inverse T, the output's weights Pm and the per-step factors, for
// every (batch row, head, chunk) at once.
//
// One block of four waves per chunk. K K^T and Q K^T (the ten lower 16 x 16
// tiles each) run on the matrix cores from halves in LDS. M = L diag(beta) is
// strictly lower, and T = (1 + M)^-1 is found by substitution, never by powers
// of M (with equal keys and no decay the powers reach 10^18 and cancel): wave w
// inverts the diagonal block w in registers, one column a lane, then takes
// block column w of T down the rows, T_iw = -T_ii sum_k M_ik T_kw, in float32
// matrix instructions, again without leaving the wave's registers.
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
  constexpr int RS = NP + 8;                          // row stride of K and Q in LDS (halves)
  constexpr int kKQ = 2 * RAW * kGdrC * RS * 2;       // bytes
  constexpr int kTP = 2 * kGdrC * kMS * 4;
  __shared__ __align__(16) char pool[kKQ > kTP ? kKQ : kTP];  // K and Q, then T and Pm
  __shared__ __align__(16) float sM[kGdrC * kMS];
  __shared__ double sC[kGdrC];
  __shared__ float sTop[4];
  __shared__ float sBeta[kGdrC], sKn[kGdrC], sQn[kGdrC], sKup[kGdrC], sQup[kGdrC];
  _Float16* sK = reinterpret_cast<_Float16*>(pool);   // [RAW][64][RS]
  _Float16* sQ = sK + RAW * kGdrC * RS;
  float* sT = reinterpret_cast<float*>(pool);         // [64][kMS]
  float* sP = sT + kGdrC * kMS;

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, m = lane & 15, g = lane >> 4;
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads);
  const int64_t item = blockIdx.x;
  const int c = static_cast<int>(item % chunks);
  const int bh = static_cast<int>(item / chunks);
  const int b = bh / H, h = bh % H, kh = h / (H / G);
  const int64_t len = gdr_row_steps(p.seqlens, b, p.seqlen);
  const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
  if (t0 >= len) return;  // behind the row's last step: nothing reads this chunk
  const int rows = static_cast<int>(len - t0 < kGdrC ? len - t0 : kGdrC);
  const int64_t row0 = static_cast<int64_t>(b) * p.seqlen + t0;

  // (1) Gates: lane t of wave 0.
  if (w == 0) {
    float ld = 0.0f, beta = 0.0f;
    if (lane < rows) {
      const int64_t at = (row0 + lane) * H + h;
      ld = gdr_log_decay(p, load_elem<BF16>(p.dt, at), p.dt_bias ? p.dt_bias[h] : 0.0f, p.A[h]);
      beta = gdr_beta(p, load_elem<BF16>(p.beta, at));
    }
    const double cs = wave_prefix(ld, lane);
    sC[lane] = cs;
    sBeta[lane] = beta;
  }

  // (2) Rows of K and Q as halves.
  gdr_stage_kq<NP, BF16, VEC>(p, row0, rows, kh, tid, sK, sQ, sKn, sQn, sKup, sQup);
  __syncthreads();

  // (3) The ten lower tiles of K K^T and Q K^T, q = w, w + 4, w + 8.
  f32x4_t pm[3];
  const double cend = sC[kGdrC - 1];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int q = w + 4 * j;
    pm[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (q >= 10) continue;
    const int ti = q == 0 ? 0 : (q < 3 ? 1 : (q < 6 ? 2 : 3));
    const int si = q - ti * (ti + 1) / 2;
    f32x4_t kk = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, qk = kk;
#pragma unroll
    for (int n = 0; n < NP; n += 32) {
      const int at = (16 * ti + m) * RS + n + 8 * g, bt = (16 * si + m) * RS + n + 8 * g;
      const half8_t bk = *reinterpret_cast<const half8_t*>(sK + bt);
      const half8_t ak = *reinterpret_cast<const half8_t*>(sK + at);
      const half8_t aq = *reinterpret_cast<const half8_t*>(sQ + at);
      kk = mfma16(ak, bk, kk);
      qk = mfma16(aq, bk, qk);
      if constexpr (RAW == 2) {
        const half8_t bl = *reinterpret_cast<const half8_t*>(sK + kGdrC * RS + bt);
        kk = mfma16(ak, bl, kk);
        qk = mfma16(aq, bl, qk);
        kk = mfma16(*reinterpret_cast<const half8_t*>(sK + kGdrC * RS + at), bk, kk);
        qk = mfma16(*reinterpret_cast<const half8_t*>(sQ + kGdrC * RS + at), bk, qk);
      }
    }
    const int s = 16 * si + m;
    const double cs = sC[s];
    const float bs = sBeta[s] * sKn[s];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * ti + 4 * g + i;
      const float dec = exp2_hw(static_cast<float>(sC[t] - cs) * kLog2e) * bs;
      sM[t * kMS + s] = t > s ? dec * sKn[t] * kk[i] : 0.0f;
      pm[j][i] = t >= s ? p.scale * dec * sQn[t] * qk[i] : 0.0f;
    }
  }
  __syncthreads();  // K and Q are done with

  // (4) Pm into LDS; the diagonal blocks' inverses (lane m: column m).
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int q = w + 4 * j;
    if (q >= 10) continue;
    const int ti = q == 0 ? 0 : (q < 3 ? 1 : (q < 6 ? 2 : 3));
    const int si = q - ti * (ti + 1) / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) sP[(16 * ti + 4 * g + i) * kMS + 16 * si + m] = pm[j][i];
  }
  {
    float x[16];
    const float* D = sM + 16 * w * kMS + 16 * w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float acc = i == m ? 1.0f : 0.0f;
#pragma unroll
      for (int k = 0; k < i; ++k) acc = fmaf(-D[i * kMS + k], x[k], acc);
      x[i] = acc;
    }
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sT[(16 * w + i) * kMS + 16 * w + m] = x[i];
    }
  }
  __syncthreads();

  // (5) Block column w of T.
  {
    f32x4_t T[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (i == w) {
#pragma unroll
        for (int r = 0; r < 4; ++r) T[i][r] = sT[(16 * i + 4 * g + r) * kMS + 16 * i + m];
      }
      if (i > w) {
        f32x4_t X = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < i; ++k) {
          if (k >= w) X = tile_product(sM + 16 * i * kMS + 16 * k, T[k], X, m, g);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) X[r] = -X[r];
        T[i] = tile_product(sT + 16 * i * kMS + 16 * i, X, T[i], m, g);
#pragma unroll
        for (int r = 0; r < 4; ++r) sT[(16 * i + 4 * g + r) * kMS + 16 * w + m] = T[i][r];
      }
    }
  }
  __syncthreads();

  // (6) Rows 16 w .. + 15 of T and Pm as halves, in the order a lane feeds them.
  float* fac = ws.fac + item * (kGdrFactors * kGdrC);
  const int t = 16 * w + m;
  // Row tile w of a matrix (or of its transpose) as halves, scaled by rows, or
  // by one power of two for the whole triangle (T: its rows all have a 1, and
  // halves reach down to 2^-38 of the largest element).
  const auto pieces = [&](const float* src, bool up, _Float16* out, float* down, bool whole, bool lo)
                          __attribute__((always_inline)) {
    float x[2][8];
    float top = 0.0f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int s = 32 * q + (e < 4 ? 4 * g + e : 12 + 4 * g + e);
        // (a block above the diagonal was never written)
        const bool in = up ? s >= t : s <= t;
        x[q][e] = in ? src[up ? s * kMS + t : t * kMS + s] : 0.0f;
        top = fmaxf(top, fabsf(x[q][e]));
      }
    }
    top = col_max(top);
    if (whole) {
      top = lanes16_max(top);
      if (lane == 0) sTop[w] = top;
      __syncthreads();
      top = fmaxf(fmaxf(sTop[0], sTop[1]), fmaxf(sTop[2], sTop[3]));
    }
    const Pow2 s = pow2_to_top(top);
    if (whole) {
      if (tid == 0) *down = s.down;
    } else if (g == 0) {
      down[t] = s.down;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (up ? (q == 0 && w >= 2) : (q == 1 && w < 2)) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[q][e] *= s.up;
      const half8_t hi = halves(x[q]);
      _Float16* at = out + (up ? gdr_frag_up(w, q) : gdr_frag(w, q)) * 2 * kGdrFragHalves + lane * 8;
      *reinterpret_cast<half8_t*>(at) = hi;
      if (lo) *reinterpret_cast<half8_t*>(at + kGdrFragHalves) = rest(x[q], hi);
    }
  };
  pieces(sT, false, ws.T + item * kGdrPieceHalves, fac + kFacEnd * kGdrC + 1, true, true);
  if constexpr (BWD) {
    pieces(sT, true, ws.Tt + item * kGdrPieceHalves, fac + kFacTt * kGdrC, false, true);
    pieces(sP, true, ws.Pt + item * kGdrPieceHalves, fac + kFacP * kGdrC, false, true);
  } else {
    pieces(sP, false, ws.Pm + item * kGdrPieceHalves, fac + kFacP * kGdrC, false, out_lo);
  }
  if (w == 0) {
    const double ct = sC[lane];
    const float into = exp2_hw(static_cast<float>(ct) * kLog2e);
    const float last = exp2_hw(static_cast<float>(cend - ct) * kLog2e);
    fac[kFacKup * kGdrC + lane] = sKup[lane];
    fac[kFacQup * kGdrC + lane] = sQup[lane];
    fac[kFacK * kGdrC + lane] = into * sKn[lane];
    fac[kFacQ * kGdrC + lane] = p.scale * into * sQn[lane];
    fac[kFacW * kGdrC + lane] = sBeta[lane] * last * sKn[lane];
    if (lane == 0) fac[kFacEnd * kGdrC] = exp2_hw(static_cast<float>(cend) * kLog2e);
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
  const unsigned blocks = static_cast<unsigned>(a.batch * a.nheads * chunks);
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
