// Gated delta rule backward, what is left once the states S, E and the
// gradients X, dE of every chunk are there (see gdr_mma.h and
// gated_delta_reverse.h): the gradients of q, k and the gates, for every chunk
// at once. Per head, with hats for the (normalised) rows and
//   L[t,s] = e^(c_t - c_s) k_t . k_s (s < t),  Pm[t,s] = scale e^(c_t - c_s) q_t . k_s beta_s
//   N1 = dY S, N2 = dE S, N3 = E X              (64 x N, contracted over the columns)
//   dP = dY E^T, M = dE E^T                     (lower triangles)
//   Gq = dP o scale e^(c_t - c_s) beta_s,  Gk = -M o e^(c_t - c_s) beta_s (s < t)
//   dq = scale e^c N1 + Gq K
//   dk = -e^c N2 + w N3 + Gk K + Gk^T K + Gq^T Q,     w_t = beta_t e^(c_end - c_t)
//   Z = dP o scale e^(c_t - c_s) q_t . k_s - M o L
//   dbeta_s = e^(c_end - c_s) k_s . N3_s + sum_t Z[t,s]
//   dc_t = scale e^c_t q_t . N1_t - e^c_t k_t . N2_t - w_t k_t . N3_t + sum_s beta_s Z[t,s] - beta_t sum_u Z[u,t]
//          (+ sum_s w_s k_s . N3_s + e^c_end <X, S> at the chunk's end)
//   d(dt A)_t = sum_{u >= t} dc_u
// One block of four waves per (batch row, query/key head, chunk); wave w has
// row tile w. The heads that share q and k are taken one after another, their
// dq and dk added in registers: no partial sums in memory, no atomics.
#include <hip/hip_runtime.h>

#include "gdr_mma.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kGS = kGdrC + 4;   // row stride of Gq and Gk in LDS (floats)
constexpr int kPS = 32 + 8;      // row stride of the staged 64 x 32 pieces (halves)

// Eight float32 of a row, zero past `count` and where !ok. vec: 16-byte loads.
__device__ __forceinline__ void load8_f32(const float* row, int e, int count, bool ok, bool vec, float (&x)[8]) {
  if (vec) {
    f32x4_t u = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, v = u;
    if (ok && e < count) u = *reinterpret_cast<const f32x4_t*>(row + e);
    if (ok && e + 4 < count) v = *reinterpret_cast<const f32x4_t*>(row + e + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = u[i], x[4 + i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ok && e + i < count ? row[e + i] : 0.0f;
  }
}

__device__ __forceinline__ void store_split(_Float16* hi_at, int lo_off, float (&x)[8], float up) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= up;
  const half8_t hi = halves(x);
  *reinterpret_cast<half8_t*>(hi_at) = hi;
  *reinterpret_cast<half8_t*>(hi_at + lo_off) = rest(x, hi);
}

// B operand of a row-major array of halves in LDS: contraction rows r0 + 8 g + 0..7, column c0 + m.
__device__ __forceinline__ half8_t column8(const _Float16* mat, int stride, int r0, int c0, int m, int g) {
  const _Float16* at = mat + (r0 + 8 * g + (m >> 2)) * stride + c0 + 4 * (m & 3);
  return __builtin_shufflevector(lds_column4(at), lds_column4(at + 4 * stride), 0, 1, 2, 3, 4, 5, 6, 7);
}

// The same of K or Q (kq_at's order).
template <int NP>
__device__ __forceinline__ half8_t kq_column8(const _Float16* mat, int r0, int c0, int m, int g) {
  const int t = r0 + 8 * g + (m >> 2), n = c0 + 4 * (m & 3);
  return __builtin_shufflevector(lds_column4(mat + kq_at<NP>(t, n)), lds_column4(mat + kq_at<NP>(t + 4, n)), 0, 1, 2, 3, 4,
                                 5, 6, 7);
}

__device__ __forceinline__ float wave_sum64(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

template <int NP, bool BF16>
__global__ __launch_bounds__(kThreads) void gdr_grads_kernel(const GatedDeltaBwdArgs a, const GdrWork ws, int chunks,
                                                             int yvec, int nvec) {
  constexpr int RAW = BF16 ? 1 : 2, RS = NP + 8, NJ = NP / 16;
  constexpr int kMat = RAW * kGdrC * NP;
  constexpr int kLo = kGdrC * NP;
  constexpr int kSX = 32 * RS;                            // halves of a staged 32 x NP piece
  constexpr int kTP = kGdrC * kPS;                        // halves of a staged 64 x 32 piece
  constexpr int kStage = (4 * kSX + 6 * kTP) * 2;         // S, X and dY, E, dE, hi and lo
  constexpr int kG = 2 * kGdrC * kGS * 4;
  __shared__ __align__(16) _Float16 sK[kMat], sQ[kMat];
  __shared__ __align__(16) char pool[kStage > kG ? kStage : kG];
  __shared__ double sC[kGdrC];
  __shared__ float sBeta[kGdrC], sKn[kGdrC], sQn[kGdrC], sKup[kGdrC], sQup[kGdrC];
  __shared__ float sRow[4][kGdrC];                        // q.N1, k.N2, k.N3, sum_s beta_s Z
  __shared__ float sCol[4][kGdrC];                        // a wave's sums of Z down the columns
  __shared__ float sDot[4];
  const GatedDeltaArgs& p = a.f;
  _Float16* sS = reinterpret_cast<_Float16*>(pool);       // [2][32][RS]
  _Float16* sX = sS + 2 * kSX;
  _Float16* sY = sX + 2 * kSX;                            // [2][64][kPS]
  _Float16* sE = sY + 2 * kTP;
  _Float16* sD = sE + 2 * kTP;
  float* sGq = reinterpret_cast<float*>(pool);            // [64][kGS]
  float* sGk = sGq + kGdrC * kGS;

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, m = lane & 15, g = lane >> 4;
  const int H = static_cast<int>(p.nheads), G = static_cast<int>(p.nkheads), r = H / G;
  const int N = static_cast<int>(p.dstate), P = static_cast<int>(p.headdim);
  const int c = static_cast<int>(blockIdx.x) % chunks;
  const int bg = static_cast<int>(blockIdx.x) / chunks;
  const int b = bg / G, kh = bg % G;
  const int64_t L = p.seqlen;
  const int64_t len = gdr_row_steps(p.seqlens, b, L);
  const int64_t t0 = static_cast<int64_t>(c) * kGdrC;
  const int64_t row0 = static_cast<int64_t>(b) * L + t0;
  const int rows = static_cast<int>(len - t0 < 0 ? 0 : (len - t0 < kGdrC ? len - t0 : kGdrC));
  const int out_rows = static_cast<int>(L - t0 < kGdrC ? L - t0 : kGdrC);
  const int64_t items = p.batch * H * static_cast<int64_t>(chunks);
  const uint32_t grow = static_cast<uint32_t>(G * N);
  const rsrc_t rdq = rows_buffer<4>(a.dq, row0 * grow + static_cast<int64_t>(kh) * N, out_rows, grow, N);
  const rsrc_t rdk = rows_buffer<4>(a.dk, row0 * grow + static_cast<int64_t>(kh) * N, out_rows, grow, N);

  f32x4_t dq[NJ], dk[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) dq[j] = dk[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  if (rows > 0) {
    const u32x4_t* K = reinterpret_cast<const u32x4_t*>(ws.K + static_cast<int64_t>(blockIdx.x) * kMat);
    const u32x4_t* Q = reinterpret_cast<const u32x4_t*>(ws.Q + static_cast<int64_t>(blockIdx.x) * kMat);
    for (int i = tid; i < kMat / 8; i += kThreads) {
      reinterpret_cast<u32x4_t*>(sK)[i] = K[i];
      reinterpret_cast<u32x4_t*>(sQ)[i] = Q[i];
    }
    const float* fac = ws.fac + ((static_cast<int64_t>(b) * H + kh * r) * chunks + c) * (kGdrFactors * kGdrC);
    if (tid < kGdrC) {
      sKn[tid] = fac[kFacKn * kGdrC + tid];
      sQn[tid] = fac[kFacQn * kGdrC + tid];
      sKup[tid] = fac[kFacKup * kGdrC + tid];
      sQup[tid] = fac[kFacQup * kGdrC + tid];
    }
  }

  for (int hh = 0; hh < r; ++hh) {
    const int h = kh * r + hh;
    const int64_t item = (static_cast<int64_t>(b) * H + h) * chunks + c;
    if (rows == 0) {  // behind the row's last step
      if (w == 0) {
        if (lane < out_rows) {
          a.ddt[(row0 + lane) * H + h] = 0.0f;
          a.dbeta[(row0 + lane) * H + h] = 0.0f;
        }
        if (lane == 0) ws.part[item] = ws.part[items + item] = 0.0f;
      }
      continue;
    }
    // Gates (wave 0; its lane t keeps the step's values for the end).
    float x = 0.0f, beta_raw = 0.0f;
    if (w == 0) {
      float ld = 0.0f, beta = 0.0f;
      if (lane < rows) {
        const int64_t at = (row0 + lane) * H + h;
        x = load_elem<BF16>(p.dt, at) + (p.dt_bias ? p.dt_bias[h] : 0.0f);
        ld = gdr_log_decay(p, load_elem<BF16>(p.dt, at), p.dt_bias ? p.dt_bias[h] : 0.0f, p.A[h]);
        beta_raw = load_elem<BF16>(p.beta, at);
        beta = gdr_beta(p, beta_raw);
      }
      sC[lane] = wave_prefix(ld, lane);
      sBeta[lane] = beta;
    }
    Pow2 top[kGdrMaxima];
    {
      const float* t = ws.top + item * kGdrMaxima * kGdrMaxSlots;
      const int slots = (P + 15) / 16 * 2;
#pragma unroll
      for (int k = 0; k < kGdrMaxima; ++k) {
        float v = 0.0f;
        for (int i = 0; i < slots; ++i) v = fmaxf(v, t[k * kGdrMaxSlots + i]);
        top[k] = pow2_to_top(v);
      }
    }

    f32x4_t n1[NJ], n2[NJ], n3[NJ], dp[4], mm[4];
#pragma unroll
    for (int j = 0; j < NJ; ++j) n1[j] = n2[j] = n3[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) dp[j] = mm[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float dot = 0.0f;  // this thread's part of <X, S>

    for (int p0 = 0; p0 < P; p0 += 32) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 32 * NP / 8 / kThreads; ++i) {
        const int e = (i * kThreads + tid) * 8, pr = e / NP, n = e % NP;
        const bool ok = p0 + pr < P;
        float s[8], xx[8];
        load8_f32(ws.S + (item * P + p0 + pr) * N, n, N, ok, nvec, s);
        load8_f32(ws.X + (item * P + p0 + pr) * N, n, N, ok, nvec, xx);
#pragma unroll
        for (int k = 0; k < 8; ++k) dot = fmaf(s[k], xx[k], dot);
        store_split(sS + pr * RS + n, kSX, s, top[kMaxS].up);
        store_split(sX + pr * RS + n, kSX, xx, top[kMaxX].up);
      }
      {
        const int t = tid >> 2, e = 8 * (tid & 3);
        const bool ok = t < rows;
        float v[8];
        load8_f32(a.dy + (row0 + t) * H * P + h * P + p0, e, P - p0, ok, yvec, v);
        store_split(sY + t * kPS + e, kTP, v, top[kMaxDY].up);
        load8_f32(a.dv + (row0 + t) * H * P + h * P + p0, e, P - p0, ok, yvec, v);
        store_split(sD + t * kPS + e, kTP, v, top[kMaxDE].up);
        load8_f32(ws.E + (item * kGdrC + t) * P + p0, e, P - p0, true, P % 4 == 0, v);
        store_split(sE + t * kPS + e, kTP, v, top[kMaxE].up);
      }
      __syncthreads();
      const int at = (16 * w + m) * kPS + 8 * g;
      const half8_t yh = *reinterpret_cast<const half8_t*>(sY + at), yl = *reinterpret_cast<const half8_t*>(sY + kTP + at);
      const half8_t eh = *reinterpret_cast<const half8_t*>(sE + at), el = *reinterpret_cast<const half8_t*>(sE + kTP + at);
      const half8_t dh = *reinterpret_cast<const half8_t*>(sD + at), dl = *reinterpret_cast<const half8_t*>(sD + kTP + at);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const half8_t sh = column8(sS, RS, 0, 16 * j, m, g), sl = column8(sS + kSX, RS, 0, 16 * j, m, g);
        const half8_t xh = column8(sX, RS, 0, 16 * j, m, g), xl = column8(sX + kSX, RS, 0, 16 * j, m, g);
        n1[j] = mfma16(yh, sh, n1[j]);
        n2[j] = mfma16(dh, sh, n2[j]);
        n3[j] = mfma16(eh, xh, n3[j]);
        n1[j] = mfma16(yh, sl, n1[j]);
        n2[j] = mfma16(dh, sl, n2[j]);
        n3[j] = mfma16(eh, xl, n3[j]);
        n1[j] = mfma16(yl, sh, n1[j]);
        n2[j] = mfma16(dl, sh, n2[j]);
        n3[j] = mfma16(el, xh, n3[j]);
      }
#pragma unroll
      for (int si = 0; si < 4; ++si) {
        if (si > w) continue;
        const int bt = (16 * si + m) * kPS + 8 * g;
        const half8_t bh = *reinterpret_cast<const half8_t*>(sE + bt), bl = *reinterpret_cast<const half8_t*>(sE + kTP + bt);
        dp[si] = mfma16(yh, bh, dp[si]);
        mm[si] = mfma16(dh, bh, mm[si]);
        dp[si] = mfma16(yh, bl, dp[si]);
        mm[si] = mfma16(dh, bl, mm[si]);
        dp[si] = mfma16(yl, bh, dp[si]);
        mm[si] = mfma16(dl, bh, mm[si]);
      }
    }
    dot = wave_sum64(dot);
    if (lane == 0) sDot[w] = dot;
    __syncthreads();  // the staged pieces are done with; Gq and Gk take their place

    const double cend = sC[kGdrC - 1];
    float ct[4], into[4], wt[4], row_z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * g + i;
      ct[i] = 0.0f;
      into[i] = exp2_hw(static_cast<float>(sC[t]) * kLog2e);
      wt[i] = sBeta[t] * exp2_hw(static_cast<float>(cend - sC[t]) * kLog2e);
      row_z[i] = 0.0f;
    }
    (void)ct;
#pragma unroll
    for (int si = 0; si < 4; ++si) {
      float col_z = 0.0f;
      const int s = 16 * si + m;
      if (si <= w) {
        f32x4_t kk = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, qk = kk;
#pragma unroll
        for (int n = 0; n < NP; n += 32) {
          const int at = kq_at<NP>(16 * w + m, n + 8 * g), bt = kq_at<NP>(16 * si + m, n + 8 * g);
          const half8_t bk = *reinterpret_cast<const half8_t*>(sK + bt);
          const half8_t ak = *reinterpret_cast<const half8_t*>(sK + at);
          const half8_t aq = *reinterpret_cast<const half8_t*>(sQ + at);
          kk = mfma16(ak, bk, kk);
          qk = mfma16(aq, bk, qk);
          if constexpr (RAW == 2) {
            const half8_t bl = *reinterpret_cast<const half8_t*>(sK + kLo + bt);
            kk = mfma16(ak, bl, kk);
            qk = mfma16(aq, bl, qk);
            kk = mfma16(*reinterpret_cast<const half8_t*>(sK + kLo + at), bk, kk);
            qk = mfma16(*reinterpret_cast<const half8_t*>(sQ + kLo + at), bk, qk);
          }
        }
        const float bs = sBeta[s], kns = sKn[s];
        const double cs = sC[s];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * w + 4 * g + i;
          const float dec = exp2_hw(static_cast<float>(sC[t] - cs) * kLog2e);
          const float u = s <= t ? dp[si][i] * (top[kMaxDY].down * top[kMaxE].down) * (p.scale * dec) : 0.0f;
          const float v = s < t ? mm[si][i] * (top[kMaxDE].down * top[kMaxE].down) * dec : 0.0f;
          const float z = u * (qk[i] * sQn[t] * kns) - v * (kk[i] * sKn[t] * kns);
          const float zz = s <= t ? z : 0.0f;  // (no product of a masked infinity)
          row_z[i] = fmaf(bs, zz, row_z[i]);
          col_z += zz;
          sGq[t * kGS + s] = u * bs;
          sGk[t * kGS + s] = -v * bs;
        }
      }
      const auto x32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(col_z), __float_as_uint(col_z), false, false);
      col_z = __uint_as_float(x32[0]) + __uint_as_float(x32[1]);
      const auto x16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(col_z), __float_as_uint(col_z), false, false);
      col_z = __uint_as_float(x16[0]) + __uint_as_float(x16[1]);
      if (g == 0) sCol[w][s] = col_z;
    }
    // Row products with N1, N2, N3, and their parts of dq and dk.
    {
      const float f1 = top[kMaxDY].down * top[kMaxS].down, f2 = top[kMaxDE].down * top[kMaxS].down;
      const float f3 = top[kMaxE].down * top[kMaxX].down;
      float r1[4] = {0.0f, 0.0f, 0.0f, 0.0f}, r2[4] = {0.0f, 0.0f, 0.0f, 0.0f}, r3[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = kq_at<NP>(16 * w + 4 * g + i, 16 * j + m);
          float kv = static_cast<float>(sK[at]), qv = static_cast<float>(sQ[at]);
          if constexpr (RAW == 2) {
            kv += static_cast<float>(sK[kLo + at]);
            qv += static_cast<float>(sQ[kLo + at]);
          }
          const float v1 = n1[j][i] * f1, v2 = n2[j][i] * f2, v3 = n3[j][i] * f3;
          r1[i] = fmaf(qv, v1, r1[i]);
          r2[i] = fmaf(kv, v2, r2[i]);
          r3[i] = fmaf(kv, v3, r3[i]);
          dq[j][i] = fmaf(p.scale * into[i], v1, dq[j][i]);
          dk[j][i] += fmaf(wt[i], v3, -into[i] * v2);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * w + 4 * g + i;
        const float q1 = lanes16_sum(r1[i]), q2 = lanes16_sum(r2[i]), q3 = lanes16_sum(r3[i]);
        const float qz = lanes16_sum(row_z[i]);
        if (m == 0) {
          sRow[0][t] = q1 * sQn[t];
          sRow[1][t] = q2 * sKn[t];
          sRow[2][t] = q3 * sKn[t];
          sRow[3][t] = qz;
        }
      }
    }
    __syncthreads();

    // dq += Gq K;  dk += Gk K + Gk^T K + Gq^T Q. The row factors of K and Q go
    // into the triangles' columns; a triangle's rows 16 w .. are halves of one scale.
    const auto product = [&](const float* G, bool up, const float* cn, const _Float16* mat, f32x4_t* out)
                             __attribute__((always_inline)) {
      const int t = 16 * w + m;
      float x8[2][8];
      float mx = 0.0f;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int s = 32 * q + 8 * g + e;
          x8[q][e] = (up ? s >= t : s <= t) ? G[up ? s * kGS + t : t * kGS + s] * cn[s] : 0.0f;
          mx = fmaxf(mx, fabsf(x8[q][e]));
        }
      }
      const Pow2 sc = pow2_to_top(lanes16_max(col_max(mx)));
      half8_t hi[2], lo[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x8[q][e] *= sc.up;
        hi[q] = halves(x8[q]);
        lo[q] = rest(x8[q], hi[q]);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (up ? (q == 0 && w >= 2) : (q == 1 && w < 2)) continue;
          const half8_t bv = kq_column8<NP>(mat, 32 * q, 16 * j, m, g);
          acc = mfma16(hi[q], bv, acc);
          acc = mfma16(lo[q], bv, acc);
          if constexpr (RAW == 2) acc = mfma16(hi[q], kq_column8<NP>(mat + kLo, 32 * q, 16 * j, m, g), acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) out[j][i] = fmaf(acc[i], sc.down, out[j][i]);
      }
    };
    product(sGq, false, sKn, sK, dq);
    product(sGk, false, sKn, sK, dk);
    product(sGk, true, sKn, sK, dk);
    product(sGq, true, sQn, sQ, dk);

    // The gates: lane t of wave 0.
    if (w == 0) {
      const double cl = sC[lane];
      const float in = exp2_hw(static_cast<float>(cl) * kLog2e);
      const float last = exp2_hw(static_cast<float>(cend - cl) * kLog2e);
      const float beta = sBeta[lane], colz = (sCol[0][lane] + sCol[1][lane]) + (sCol[2][lane] + sCol[3][lane]);
      const float r3 = sRow[2][lane];
      const float w3 = beta * last * r3;
      float dc = p.scale * in * sRow[0][lane] - in * sRow[1][lane] - w3 + sRow[3][lane] - beta * colz;
      const float dbeta = fmaf(last, r3, colz);
      // sum over the steps from t on, the end's own part with the last one
      const float at_end = wave_sum64(w3) + exp2_hw(static_cast<float>(cend) * kLog2e) *
                                                ((sDot[0] + sDot[1]) + (sDot[2] + sDot[3]));
      double suffix = dc;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_down(suffix, d);
        if (lane + d < 64) suffix += o;
      }
      const float A = p.A[h];
      const float dt = p.dt_softplus ? softplus_f(x) : x;
      float dg = static_cast<float>(suffix + static_cast<double>(at_end));
      if (lane >= rows || dt * A < kGdrMinLogDecay) dg = 0.0f;  // behind the end; where the decay was cut off
      float ddt = dg * A;
      if (p.dt_softplus) ddt *= sigmoid_f(x);
      float db = dbeta;
      if (p.beta_sigmoid) db *= beta * (1.0f - beta);
      if (lane < out_rows) {
        a.ddt[(row0 + lane) * H + h] = lane < rows ? ddt : 0.0f;
        a.dbeta[(row0 + lane) * H + h] = lane < rows ? db : 0.0f;
      }
      const float da = wave_sum64(lane < rows && dg != 0.0f ? dg * dt : 0.0f);
      const float dbias = wave_sum64(lane < rows ? ddt : 0.0f);
      if (lane == 0) {
        ws.part[item] = da;
        ws.part[items + item] = dbias;
      }
    }
    __syncthreads();
  }

  // Through the norms: d = n (dhat - hat (hat . dhat)), hat = raw n.
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 16 * w + 4 * g + i;
    float sq = 0.0f, sk = 0.0f, qv[NJ], kv[NJ];
    const bool on = t < rows;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int at = kq_at<NP>(t, 16 * j + m);
      qv[j] = kv[j] = 0.0f;
      if (rows > 0 && p.qk_l2norm) {
        qv[j] = static_cast<float>(sQ[at]);
        kv[j] = static_cast<float>(sK[at]);
        if constexpr (RAW == 2) {
          qv[j] += static_cast<float>(sQ[kLo + at]);
          kv[j] += static_cast<float>(sK[kLo + at]);
        }
        qv[j] *= sQn[t];
        kv[j] *= sKn[t];
        sq = fmaf(qv[j], dq[j][i], sq);
        sk = fmaf(kv[j], dk[j][i], sk);
      }
    }
    float nq = 1.0f, nk = 1.0f;
    if (rows > 0 && p.qk_l2norm) {
      sq = lanes16_sum(sq);
      sk = lanes16_sum(sk);
      nq = sQn[t] * sQup[t];
      nk = sKn[t] * sKup[t];
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = 16 * j + m;
      const uint32_t off = n < N ? (static_cast<uint32_t>(t) * grow + static_cast<uint32_t>(n)) * 4 : kOutOfRange;
      buffer_store_f32<false>(on ? nq * (dq[j][i] - qv[j] * sq) : 0.0f, rdq, off);
      buffer_store_f32<false>(on ? nk * (dk[j][i] - kv[j] * sk) : 0.0f, rdk, off);
    }
  }
}

// dA[h] and ddt_bias[h]: the items' parts, added in a fixed order (each thread
// every 256th of a head's batch rows and chunks, then a tree).
__global__ __launch_bounds__(kThreads) void gdr_gate_sums_kernel(const float* __restrict__ part, int64_t batch, int H,
                                                                 int64_t chunks, float* __restrict__ dA,
                                                                 float* __restrict__ dbias) {
  __shared__ float sums[2][kThreads];
  const int h = blockIdx.x, tid = threadIdx.x;
  const int64_t n = batch * chunks, items = n * H;
  float u = 0.0f, v = 0.0f;
  for (int64_t i = tid; i < n; i += kThreads) {
    const int64_t at = ((i / chunks) * H + h) * chunks + i % chunks;
    u += part[at];
    v += part[items + at];
  }
  sums[0][tid] = u;
  sums[1][tid] = v;
  __syncthreads();
  for (int s = kThreads / 2; s > 0; s >>= 1) {
    if (tid < s) {
      sums[0][tid] += sums[0][tid + s];
      sums[1][tid] += sums[1][tid + s];
    }
    __syncthreads();
  }
  if (tid == 0) {
    dA[h] = sums[0][0];
    if (dbias != nullptr) dbias[h] = sums[1][0];
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int launch_gdr_grads(const GatedDeltaBwdArgs& a, const GdrWork& ws, int64_t chunks, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int n = static_cast<int>(chunks);
  if (n > 0) {
    const unsigned blocks = static_cast<unsigned>(a.f.batch * a.f.nkheads * chunks);
    const int yvec = a.f.headdim % 4 == 0 && on16(a.dy) && on16(a.dv), nvec = a.f.dstate % 4 == 0;
    const auto types = [&](auto np, auto bf16) {
      constexpr int NP = decltype(np)::value;
      constexpr bool BF16 = decltype(bf16)::value;
      gdr_grads_kernel<NP, BF16><<<blocks, kThreads, 0, st>>>(a, ws, n, yvec, nvec);
    };
    const auto width = [&](auto np) { a.f.in_bf16 ? types(np, std::true_type{}) : types(np, std::false_type{}); };
    if (a.f.dstate <= 64) {
      width(std::integral_constant<int, 64>{});
    } else {
      width(std::integral_constant<int, 128>{});
    }
    if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  }
  gdr_gate_sums_kernel<<<static_cast<unsigned>(a.f.nheads), kThreads, 0, st>>>(
      ws.part, n > 0 ? a.f.batch : 0, static_cast<int>(a.f.nheads), n > 0 ? chunks : 1, a.dA, a.ddt_bias);
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
