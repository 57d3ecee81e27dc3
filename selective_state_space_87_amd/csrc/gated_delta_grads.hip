// Gated delta rule backward, what is left once the states S, E and the
// gradients X, dE of every chunk are there (see gdr_mma.h and
// gated_delta_reverse.hip): the gradients of q, k and the gates, for every chunk
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
// Signs (see gdr_mma.h): every other 16 columns n of S and X, and every other row
// of E, are taken negative, so that the products' errors cancel in the sums over n
// and over steps; X comes with every other 16 of its rows p negative already.
// Gq and Gk are kept with the row factors of both their sides (those of k on
// the columns, of q or k on the rows) and taken out of the products' rows again:
// one set of halves, read by rows and, transposed by the LDS, by columns, serves
// Gq K and Gq^T Q, and one Gk K and Gk^T K.
// One block of eight waves per (batch row, query/key head, chunk); wave w has
// row tile w % 4 and half w / 4 of the N columns (and of dP and M: the one or
// the other). The heads that share q and k are taken one after another, their
// dq and dk added in registers: no partial sums in memory, no atomics.
// Measured at (2, 4096, 16 heads of 128 x 128), bfloat16 inputs, 0.54 GB in and
// 0.14 GB out: 226 us, one block a CU. (Four waves a block: 600 us, for the 192
// registers of a wave's accumulators left none for operands. Gq and Gk in
// float32, made into halves once for each of the four products: 30 us more. Gates
// and scales read where they are used: 17 us more. Addresses kept over the heads,
// which spilled: 10 us more.) While the pieces of S and X are read, a quarter of
// the time, HBM gives 4.3 TB/s; between, it waits for the products.
#include <hip/hip_runtime.h>

#include "gdr_mma.h"

namespace ssm {

namespace {

constexpr int kThreads = 512;
constexpr int kGS = kGdrC + 8;   // row stride of Gq and Gk in LDS (halves)
constexpr int kPS = 32 + 8;      // row stride of the staged 64 x 32 pieces (halves)

// Elements e .. e+7 of a float32 row that starts `row` elements into the
// buffer; zero past `count` and where !ok. FAST: rows on 16-byte boundaries,
// count a multiple of 4. (No branch: a conditional load is waited for where
// the branches join.)
template <bool FAST>
__device__ __forceinline__ void load8_f32(rsrc_t r, uint32_t row, int e, int count, bool ok, float (&x)[8]) {
  const uint32_t at = (row + static_cast<uint32_t>(e)) * 4;
  if constexpr (FAST) {
    const u32x4_t u = __builtin_amdgcn_raw_buffer_load_b128(r, ok && e < count ? at : kOutOfRange, 0, 0);
    const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, ok && e + 4 < count ? at + 16 : kOutOfRange, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]), x[4 + i] = __uint_as_float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          r, ok && e + i < count ? at + static_cast<uint32_t>(4 * i) : kOutOfRange, 0, 0));
    }
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

// A value that all lanes share, in a scalar register.
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

template <typename T>
__device__ __forceinline__ T wave_sum64(T v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// The factors of a chunk's 64 rows of K or Q, a lane each. unit: the power of
// two of the largest (down: that power, up: its inverse). Rows whose factor is
// under 2^-8 of it (a key of nothing has one of 2^-113) are lifted by a power of
// two there, and their halves lowered: Gq and Gk, kept with the factors of
// their rows and columns, then hold every row of the products to 2^-38 2^16 of
// the largest. The halves themselves stay as exact as they were for rows down
// to 2^-24 of the largest.
__device__ __forceinline__ Pow2 row_lift(float f, Pow2& unit) {
  const int e = static_cast<int>(__float_as_uint(f) >> 23) & 255;
  const int top = static_cast<int>(__float_as_uint(uniform(lanes16_max(col_max(f)))) >> 23) & 255;
  const int u = top < 8 ? 8 : (top > 246 ? 246 : top);
  unit = Pow2{__uint_as_float(static_cast<uint32_t>(254 - u) << 23), __uint_as_float(static_cast<uint32_t>(u) << 23)};
  int j = top - 8 - e;
  j = j < 0 ? 0 : (j > 126 ? 126 : j);
  return Pow2{__uint_as_float(static_cast<uint32_t>(127 + j) << 23), __uint_as_float(static_cast<uint32_t>(127 - j) << 23)};
}

template <int NP, bool BF16, bool FAST>
__global__ __launch_bounds__(kThreads) void gdr_grads_kernel(const GatedDeltaBwdArgs a, const GdrWork ws, int chunks) {
  constexpr int RAW = BF16 ? 1 : 2, RS = NP + 8, NJ = NP / 32;  // NJ: column tiles of a wave
  constexpr int kMat = RAW * kGdrC * NP;
  constexpr int kLo = kGdrC * NP;
  constexpr int kSX = 32 * RS;                            // halves of a staged 32 x NP piece
  constexpr int kTP = kGdrC * kPS;                        // halves of a staged 64 x 32 piece
  constexpr int kStage = (4 * kSX + 6 * kTP) * 2;         // S, X and dY, E, dE, hi and lo
  constexpr int kGP = kGdrC * kGS;                        // halves of a plane of Gq or Gk
  constexpr int kG = 4 * kGP * 2;                         // Gq and Gk, hi and lo
  __shared__ __align__(16) _Float16 sK[kMat], sQ[kMat];
  __shared__ __align__(16) char pool[kStage > kG ? kStage : kG];
  __shared__ double sC[kGdrC];
  __shared__ float sBeta[kGdrC], sKn[kGdrC], sQn[kGdrC], sKup[kGdrC], sQup[kGdrC];
  __shared__ float sRow[3][2][kGdrC];                     // q.N1, k.N2, k.N3 (half the columns each)
  __shared__ double sRowZ[2][kGdrC];                      // sum_s beta_s Z (of either term of Z)
  __shared__ double sCol[8][kGdrC];                       // a wave's sums of Z down the columns
  __shared__ float sDot[8], sTop[8];
  const GatedDeltaArgs& p = a.f;
  _Float16* sS = reinterpret_cast<_Float16*>(pool);       // [2][32][RS]
  _Float16* sX = sS + 2 * kSX;
  _Float16* sY = sX + 2 * kSX;                            // [2][64][kPS]
  _Float16* sE = sY + 2 * kTP;
  _Float16* sD = sE + 2 * kTP;
  _Float16* sGq = reinterpret_cast<_Float16*>(pool);      // [2][64][kGS]
  _Float16* sGk = sGq + 2 * kGP;

  const int tid = threadIdx.x, lane = tid & 63;
  const int w8 = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w = w8 & 3, hf = w8 >> 2;                     // row tile, half
  const int c0 = hf * (NP / 2);                           // the wave's first column
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

  Pow2 kunit, qunit;
  if (rows > 0) {
    const half8_t* K = reinterpret_cast<const half8_t*>(ws.K + static_cast<int64_t>(blockIdx.x) * kMat);
    const half8_t* Q = reinterpret_cast<const half8_t*>(ws.Q + static_cast<int64_t>(blockIdx.x) * kMat);
    const float* fac = ws.fac + ((static_cast<int64_t>(b) * H + kh * r) * chunks + c) * (kGdrFactors * kGdrC);
    const float kn = fac[kFacKn * kGdrC + lane], qn = fac[kFacQn * kGdrC + lane];
    const float kup = fac[kFacKup * kGdrC + lane], qup = fac[kFacQup * kGdrC + lane];
    half8_t kv[kMat / 8 / kThreads], qv[kMat / 8 / kThreads];
#pragma unroll
    for (int i = 0; i < kMat / 8 / kThreads; ++i) kv[i] = K[i * kThreads + tid], qv[i] = Q[i * kThreads + tid];
    const Pow2 kf = row_lift(kn, kunit), qf = row_lift(qn, qunit);
#pragma unroll
    for (int i = 0; i < kMat / 8 / kThreads; ++i) {
      const int at = i * kThreads + tid, t = at * 8 % (kGdrC * NP) / NP;
      reinterpret_cast<half8_t*>(sK)[at] = kv[i] * static_cast<_Float16>(__shfl(kf.down, t));
      reinterpret_cast<half8_t*>(sQ)[at] = qv[i] * static_cast<_Float16>(__shfl(qf.down, t));
    }
    if (tid < kGdrC) {
      sKn[tid] = kn * kf.up;
      sQn[tid] = qn * qf.up;
      sKup[tid] = kup * kf.down;
      sQup[tid] = qup * qf.down;
    }
  }

  for (int hh = 0; hh < r; ++hh) {
    // The lane's place, made anew for every head as far as the compiler can
    // tell: it would else keep every LDS address and mask of the body in
    // registers across the heads (125 of them spilled).
    const int place = anew(lane), m = place & 15, g = place >> 4;
    const int h = kh * r + hh;
    const int64_t item = (static_cast<int64_t>(b) * H + h) * chunks + c;
    if (rows == 0) {  // behind the row's last step
      if (w8 == 0) {
        if (lane < out_rows) {
          a.ddt[(row0 + lane) * H + h] = 0.0f;
          a.dbeta[(row0 + lane) * H + h] = 0.0f;
        }
        if (lane == 0) ws.part[item] = ws.part[items + item] = 0.0;
      }
      continue;
    }
    // 32 columns of S, X, dY, E, dE at a time, the next ones in flight in
    // registers: a piece of S and X a thread, a piece of dY or dE, half a piece of E.
    constexpr int kSXT = 32 * NP / 8 < kThreads ? 1 : 32 * NP / 8 / kThreads;
    float fs[kSXT][8], fx[kSXT][8], fy[8], fe[8];
    const int trow = (tid >> 2) & 63, tcol = 8 * (tid & 3);
    const uint32_t yrow = static_cast<uint32_t>(H * P);
    const rsrc_t rs = raw_buffer(ws.S + item * P * N, static_cast<uint32_t>(P * N * 4));
    const rsrc_t rx = raw_buffer(ws.X + item * P * N, static_cast<uint32_t>(P * N * 4));
    const rsrc_t re = raw_buffer(ws.E + item * kGdrC * P, static_cast<uint32_t>(kGdrC * P * 4));
    const rsrc_t ry = rows_buffer<4>(hf == 0 ? a.dy : a.dv, row0 * yrow + static_cast<int64_t>(h) * P, rows, yrow, P);
    const auto fetch = [&](int p0) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kSXT; ++i) {
        const int e = (i * kThreads + tid) * 8 % (32 * NP), pr = e / NP, n = e % NP;
        const bool ok = p0 + pr < P;
        load8_f32<FAST>(rs, static_cast<uint32_t>((p0 + pr) * N), n, N, ok, fs[i]);
        load8_f32<FAST>(rx, static_cast<uint32_t>((p0 + pr) * N), n, N, ok, fx[i]);
      }
      load8_f32<FAST>(ry, static_cast<uint32_t>(trow) * yrow + static_cast<uint32_t>(p0), tcol, P - p0, trow < rows, fy);
      load8_f32<FAST>(re, static_cast<uint32_t>(trow * P + p0), tcol, P - p0, true, fe);
    };
    // What the gates and the scales need, then the first pieces: loads in no branch.
    const int64_t gate_at = (row0 + (place < rows ? place : rows - 1)) * H + h;
    const float dt_raw = load_elem<BF16>(p.dt, gate_at), beta_raw = load_elem<BF16>(p.beta, gate_at);
    const float dt_bias = p.dt_bias ? p.dt_bias[h] : 0.0f, A = p.A[h];
    float tops[kGdrMaxima];
    {
      const float* t = ws.top + item * kGdrMaxima * kGdrMaxSlots;
      const int slots = (P + 15) / 16 * 2, slot = (place & 31) < slots ? place & 31 : slots - 1;
#pragma unroll
      for (int k = 0; k < kGdrMaxima; ++k) tops[k] = t[k * kGdrMaxSlots + slot];
    }
    fetch(0);
    // Gates (wave 0; its lane t keeps the step's values for the end).
    const float x = dt_raw + dt_bias;
    if (w8 == 0) {
      const float ld = place < rows ? gdr_log_decay(p, dt_raw, dt_bias, A) : 0.0f;
      sC[place] = wave_prefix(static_cast<double>(ld) * kLog2eD, place);
      sBeta[place] = place < rows ? gdr_beta(p, beta_raw) : 0.0f;
    }
    Pow2 top[kGdrMaxima];
#pragma unroll
    for (int k = 0; k < kGdrMaxima; ++k) top[k] = pow2_to_top(uniform(lanes16_max(col_max(tops[k]))));

    f32x4_t n1[NJ], n2[NJ], n3[NJ], tri[4];
#pragma unroll
    for (int j = 0; j < NJ; ++j) n1[j] = n2[j] = n3[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) tri[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float dot = 0.0f;  // this thread's part of <X, S>

    for (int p0 = 0; p0 < P; p0 += 32) {
      const int at_tid = anew(tid);  // (for the signs, that they are not kept in registers)
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kSXT; ++i) {
        const int e = (i * kThreads + tid) * 8 % (32 * NP), pr = e / NP, n = e % NP;
        const int from = (i * kThreads + at_tid) * 8 % (32 * NP), sp = from / NP >> 4, sn = from % NP >> 4;
        if (32 * NP / 8 >= kThreads || tid < 32 * NP / 8) {
#pragma unroll
          for (int k = 0; k < 8; ++k) dot = fmaf(flip(fs[i][k], sp), fx[i][k], dot);
        }
        // (with 64 states two threads have, and write, the same piece)
        store_split(sS + pr * RS + n, kSX, fs[i], flip(top[kMaxS].up, sn));
        store_split(sX + pr * RS + n, kSX, fx[i], flip(top[kMaxX].up, sn ^ sp));
      }
      store_split((hf == 0 ? sY : sD) + trow * kPS + tcol, kTP, fy, top[hf == 0 ? kMaxDY : kMaxDE].up);
      if (hf == 0) store_split(sE + trow * kPS + tcol, kTP, fe, flip(top[kMaxE].up, at_tid >> 2));
      __syncthreads();
      fetch(p0 + 32);  // (past the last columns: zeros)
      const int at = (16 * w + m) * kPS + 8 * g;
      const auto two = [&](const _Float16* q, half8_t& hi, half8_t& lo) __attribute__((always_inline)) {
        hi = *reinterpret_cast<const half8_t*>(q);
        lo = *reinterpret_cast<const half8_t*>(q + kTP);
      };
      half8_t yh, yl, eh, el, dh, dl;
      two(sY + at, yh, yl);
      two(sE + at, eh, el);
      two(sD + at, dh, dl);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const half8_t sh = column8(sS, RS, 0, c0 + 16 * j, m, g), sl = column8(sS + kSX, RS, 0, c0 + 16 * j, m, g);
        const half8_t xh = column8(sX, RS, 0, c0 + 16 * j, m, g), xl = column8(sX + kSX, RS, 0, c0 + 16 * j, m, g);
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
      const half8_t lh = hf == 0 ? yh : dh, ll = hf == 0 ? yl : dl;
#pragma unroll
      for (int si = 0; si < 4; ++si) {
        if (si > w) continue;
        half8_t bh, bl;
        two(sE + (16 * si + m) * kPS + 8 * g, bh, bl);
        tri[si] = mfma16(lh, bh, tri[si]);
        tri[si] = mfma16(lh, bl, tri[si]);
        tri[si] = mfma16(ll, bh, tri[si]);
      }
    }
    dot = wave_sum64(dot);
    if (place == 0) sDot[w8] = dot;
    __syncthreads();  // the staged pieces are done with; Gq and Gk take their place

    const double cend = sC[kGdrC - 1];
    float into[4], wt[4];
    double row_z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * g + i;
      into[i] = exp2_hw(static_cast<float>(sC[t]));
      wt[i] = sBeta[t] * exp2_hw(static_cast<float>(cend - sC[t]));
      row_z[i] = 0.0;
    }
    // Gq and the first term of Z (half 0), Gk and the second (half 1).
    {
      const _Float16* left = hf == 0 ? sQ : sK;
      const float* ln = hf == 0 ? sQn : sKn;
      const float lup = hf == 0 ? qunit.up : kunit.up, whole = (hf == 0 ? qunit.down : kunit.down) * kunit.down;
      const float unit = flip(hf == 0 ? top[kMaxDY].down * top[kMaxE].down * p.scale : -(top[kMaxDE].down * top[kMaxE].down), m);
      float mx = 0.0f, lnt[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) lnt[i] = ln[16 * w + 4 * g + i] * lup;
#pragma unroll
      for (int si = 0; si < 4; ++si) {
        double col_z = 0.0;
        const int s = 16 * si + m;
        if (si <= w) {
          f32x4_t xk = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};  // q_t . k_s or k_t . k_s
#pragma unroll
          for (int n = 0; n < NP; n += 32) {
            const int at = kq_at<NP>(16 * w + m, n + 8 * g), bt = kq_at<NP>(16 * si + m, n + 8 * g);
            const half8_t bk = *reinterpret_cast<const half8_t*>(sK + bt);
            const half8_t al = *reinterpret_cast<const half8_t*>(left + at);
            xk = mfma16(al, bk, xk);
            if constexpr (RAW == 2) {
              xk = mfma16(al, *reinterpret_cast<const half8_t*>(sK + kLo + bt), xk);
              xk = mfma16(*reinterpret_cast<const half8_t*>(left + kLo + at), bk, xk);
            }
          }
          const float bs = sBeta[s], kns = sKn[s] * kunit.up;
          const double cs = sC[s];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 16 * w + 4 * g + i;
            const bool in = si < w || (hf == 0 ? s <= t : s < t);
            const float dec = exp2_hw(static_cast<float>(sC[t] - cs)) * (lnt[i] * kns);
            const float u = in ? tri[si][i] * unit * dec : 0.0f;
            const float z = in ? u * (xk[i] * whole) : 0.0f;  // (no product of a masked infinity)
            row_z[i] = fma(static_cast<double>(bs), static_cast<double>(z), row_z[i]);
            col_z += z;
            tri[si][i] = u * bs;
            mx = fmaxf(mx, fabsf(tri[si][i]));
          }
        } else {
          tri[si] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
        col_z += __shfl_xor(col_z, 32);
        col_z += __shfl_xor(col_z, 16);
        if (g == 0) sCol[w8][s] = col_z;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        double z = row_z[i];
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) z += __shfl_xor(z, d);
        if (m == 0) sRowZ[hf][16 * w + 4 * g + i] = z;
      }
      mx = lanes16_max(col_max(mx));
      if (place == 0) sTop[w8] = mx;
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
          const int at = kq_at<NP>(16 * w + 4 * g + i, c0 + 16 * j + m);
          float kv = static_cast<float>(sK[at]), qv = static_cast<float>(sQ[at]);
          if constexpr (RAW == 2) {
            kv += static_cast<float>(sK[kLo + at]);
            qv += static_cast<float>(sQ[kLo + at]);
          }
          const float v1 = n1[j][i] * (j & 1 ? -f1 : f1), v2 = n2[j][i] * (j & 1 ? -f2 : f2);
          const float v3 = n3[j][i] * ((i ^ j) & 1 ? -f3 : f3);
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
        if (m == 0) {
          sRow[0][hf][t] = q1 * sQn[t];
          sRow[1][hf][t] = q2 * sKn[t];
          sRow[2][hf][t] = q3 * sKn[t];
        }
      }
    }
    __syncthreads();

    // dq += Gq K;  dk += Gk K + Gk^T K + Gq^T Q.
    Pow2 sg[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sg[k] = pow2_to_top(fmaxf(fmaxf(sTop[4 * k], sTop[4 * k + 1]), fmaxf(sTop[4 * k + 2], sTop[4 * k + 3])));
    }
    {
      // the wave's tiles of its triangle, and the zeros right of an even
      // diagonal tile (pieces are two tiles wide)
      _Float16* out = hf == 0 ? sGq : sGk;
      const float up = hf == 0 ? sg[0].up : sg[1].up;
#pragma unroll
      for (int si = 0; si < 4; ++si) {
        if (si > (w | 1)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = tri[si][i] * up;
          const _Float16 hi = static_cast<_Float16>(v);
          const int at = (16 * w + 4 * g + i) * kGS + 16 * si + m;
          out[at] = hi;
          out[kGP + at] = static_cast<_Float16>(v - static_cast<float>(hi));
        }
      }
    }
    __syncthreads();
    {
      f32x4_t aq[NJ], ak[NJ], ag[NJ];  // Gq K; Gk K + Gk^T K; Gq^T Q
#pragma unroll
      for (int j = 0; j < NJ; ++j) aq[j] = ak[j] = ag[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool low = 2 * q <= w, upp = 2 * q + 1 >= w;  // (of the wave)
        const int at = (16 * w + m) * kGS + 32 * q + 8 * g;
        half8_t bk[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) bk[j] = kq_column8<NP>(sK, 32 * q, c0 + 16 * j, m, g);
        const auto times_k = [&](half8_t hi, half8_t lo, f32x4_t* acc) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            acc[j] = mfma16(hi, bk[j], acc[j]);
            acc[j] = mfma16(lo, bk[j], acc[j]);
            if constexpr (RAW == 2) acc[j] = mfma16(hi, kq_column8<NP>(sK + kLo, 32 * q, c0 + 16 * j, m, g), acc[j]);
          }
        };
        if (low) {
          times_k(*reinterpret_cast<const half8_t*>(sGq + at), *reinterpret_cast<const half8_t*>(sGq + kGP + at), aq);
          times_k(*reinterpret_cast<const half8_t*>(sGk + at), *reinterpret_cast<const half8_t*>(sGk + kGP + at), ak);
        }
        if (upp) {
          times_k(column8(sGk, kGS, 32 * q, 16 * w, m, g), column8(sGk + kGP, kGS, 32 * q, 16 * w, m, g), ak);
          const half8_t hi = column8(sGq, kGS, 32 * q, 16 * w, m, g), lo = column8(sGq + kGP, kGS, 32 * q, 16 * w, m, g);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const half8_t bq = kq_column8<NP>(sQ, 32 * q, c0 + 16 * j, m, g);
            ag[j] = mfma16(hi, bq, ag[j]);
            ag[j] = mfma16(lo, bq, ag[j]);
            if constexpr (RAW == 2) ag[j] = mfma16(hi, kq_column8<NP>(sQ + kLo, 32 * q, c0 + 16 * j, m, g), ag[j]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * w + 4 * g + i;
        const float iq = kunit.down * sg[0].down / (sQn[t] * qunit.up), ik = 1.0f / (sKn[t] * kunit.up);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          dq[j][i] = fmaf(aq[j][i], iq, dq[j][i]);
          dk[j][i] = fmaf(ik, fmaf(ag[j][i], qunit.down * sg[0].down, ak[j][i] * (kunit.down * sg[1].down)), dk[j][i]);
        }
      }
    }

    // The gates: lane t of wave 0.
    if (w8 == 0) {
      // Summed in double, Z's sums over rows and columns above as well: what a pair
      // of steps on the same side of t adds to one of them it takes from the other,
      // to the bit, and does not leave 64 roundings in d(dt A)_t, which then all
      // point one way in dA. (In float32: ddt off by 6.4e-7, now 2.7e-7; 9 us less.)
      const int t = anew(lane);  // (its addresses are not kept from one head to the next)
      const double cl = sC[t];
      const float in = exp2_hw(static_cast<float>(cl));
      const float last = exp2_hw(static_cast<float>(cend - cl));
      const float beta = sBeta[t];
      double colz = 0.0, dots = 0.0;
#pragma unroll
      for (int k = 0; k < 8; ++k) colz += sCol[k][t], dots += sDot[k];
      const auto row = [&](int k) { return sRow[k][0][t] + sRow[k][1][t]; };
      const float r3 = row(2);
      const double w3 = static_cast<double>(beta * last) * r3;
      const double dc = static_cast<double>(p.scale * in) * row(0) - static_cast<double>(in) * row(1) - w3 +
                        (sRowZ[0][t] + sRowZ[1][t]) - static_cast<double>(beta) * colz;
      const float dbeta = fmaf(last, r3, static_cast<float>(colz));
      // sum over the steps from t on, the end's own part with the last one
      const double at_end = wave_sum64(w3) + static_cast<double>(exp2_hw(static_cast<float>(cend))) * dots;
      double suffix = dc;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_down(suffix, d);
        if (t + d < 64) suffix += o;
      }
      const float dt = p.dt_softplus ? gdr_softplus(x) : x;
      float dg = static_cast<float>(suffix + at_end);
      if (t >= rows || dt * A < kGdrMinLogDecay) dg = 0.0f;  // behind the end; where the decay was cut off
      float ddt = dg * A;
      if (p.dt_softplus) ddt *= sigmoid_f(x);
      float db = dbeta;
      // (1 - beta of the rounded beta would be 0 from a raw strength of 17 on)
      if (p.beta_sigmoid) db *= sigmoid_f(beta_raw) * sigmoid_f(-beta_raw);
      if (t < out_rows) {
        const int64_t at = (row0 + t) * H + h;
        a.ddt[at] = t < rows ? ddt : 0.0f;
        a.dbeta[at] = t < rows ? db : 0.0f;
      }
      // (In double to the last sum: terms of thousands of steps cancel.)
      const double da = wave_sum64(t < rows && dg != 0.0f ? static_cast<double>(dg) * dt : 0.0);
      const double dbias = wave_sum64(t < rows ? static_cast<double>(ddt) : 0.0);
      if (t == 0) {
        ws.part[item] = da;
        ws.part[items + item] = dbias;
      }
    }
    __syncthreads();
  }

  const int m = lane & 15, g = lane >> 4;
  // Through the norms: d = n (dhat - hat (hat . dhat)), hat = raw n.
  const bool norm = rows > 0 && p.qk_l2norm;
  if (norm) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * g + i;
      float sq = 0.0f, sk = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int at = kq_at<NP>(t, c0 + 16 * j + m);
        float qv = static_cast<float>(sQ[at]), kv = static_cast<float>(sK[at]);
        if constexpr (RAW == 2) {
          qv += static_cast<float>(sQ[kLo + at]);
          kv += static_cast<float>(sK[kLo + at]);
        }
        sq = fmaf(qv, dq[j][i], sq);
        sk = fmaf(kv, dk[j][i], sk);
      }
      sq = lanes16_sum(sq);
      sk = lanes16_sum(sk);
      if (m == 0) {
        sRow[0][hf][t] = sq * sQn[t];
        sRow[1][hf][t] = sk * sKn[t];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 16 * w + 4 * g + i;
    const bool on = t < rows;
    float fq = 0.0f, fk = 0.0f, nq = 1.0f, nk = 1.0f;
    if (norm) {
      fq = (sRow[0][0][t] + sRow[0][1][t]) * sQn[t];
      fk = (sRow[1][0][t] + sRow[1][1][t]) * sKn[t];
      nq = sQn[t] * sQup[t];
      nk = sKn[t] * sKup[t];
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = c0 + 16 * j + m;
      float vq = dq[j][i], vk = dk[j][i];
      if (norm) {
        const int at = kq_at<NP>(t, n);
        float qv = static_cast<float>(sQ[at]), kv = static_cast<float>(sK[at]);
        if constexpr (RAW == 2) {
          qv += static_cast<float>(sQ[kLo + at]);
          kv += static_cast<float>(sK[kLo + at]);
        }
        vq = nq * fmaf(-qv, fq, vq);
        vk = nk * fmaf(-kv, fk, vk);
      }
      const uint32_t off = n < N ? (static_cast<uint32_t>(t) * grow + static_cast<uint32_t>(n)) * 4 : kOutOfRange;
      buffer_store_f32<false>(on ? vq : 0.0f, rdq, off);
      buffer_store_f32<false>(on ? vk : 0.0f, rdk, off);
    }
  }
}

// dA[h] and ddt_bias[h]: the items' parts, added in a fixed order (each thread
// every 512th of a head's batch rows and chunks, then a tree) and rounded once.
__global__ __launch_bounds__(kThreads) void gdr_gate_sums_kernel(const double* __restrict__ part, int64_t batch, int H,
                                                                 int64_t chunks, float* __restrict__ dA,
                                                                 float* __restrict__ dbias) {
  __shared__ double sums[2][kThreads];
  const int h = blockIdx.x, tid = threadIdx.x;
  const int64_t n = batch * chunks, items = n * H;
  double u = 0.0, v = 0.0;
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
    dA[h] = static_cast<float>(sums[0][0]);
    if (dbias != nullptr) dbias[h] = static_cast<float>(sums[1][0]);
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int launch_gdr_grads(const GatedDeltaBwdArgs& a, const GdrWork& ws, int64_t chunks, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int n = static_cast<int>(chunks);
  if (n > 0) {
    const unsigned blocks = static_cast<unsigned>(a.f.batch * a.f.nkheads * chunks);
    const bool fast = a.f.headdim % 4 == 0 && a.f.dstate % 4 == 0 && on16(a.dy) && on16(a.dv);
    const auto types = [&](auto np, auto bf16) {
      constexpr int NP = decltype(np)::value;
      constexpr bool BF16 = decltype(bf16)::value;
      fast ? gdr_grads_kernel<NP, BF16, true><<<blocks, kThreads, 0, st>>>(a, ws, n)
           : gdr_grads_kernel<NP, BF16, false><<<blocks, kThreads, 0, st>>>(a, ws, n);
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
