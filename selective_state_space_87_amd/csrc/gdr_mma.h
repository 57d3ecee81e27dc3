// The chunked form of the gated delta rule: operand precision, layouts and
// workspace shared by its kernels (gfx950).
//
// A sequence is cut into chunks of 64 steps. With c_t the sum of the log decays
// of a chunk's steps up to t, S the state entering the chunk, and row t of K, Q,
// V the step's k, q, v:
//   E  = T (V - diag(e^c) K S),      T = (1 + L diag(beta))^-1,
//        L[t,s] = e^(c_t - c_s) k_t . k_s   for s < t
//   Y  = scale diag(e^c) Q S + Pm E, Pm[t,s] = scale e^(c_t - c_s) q_t . k_s beta_s  for s <= t
//   S' = e^(c_end) S + K^T diag(beta e^(c_end - c)) E
// where row s of E is the error e_s of step s. T and Pm do not depend on the
// state: one kernel makes them for all chunks at once, another walks a head's
// chunks in order.
//
// Operands of the matrix cores. The state has to come out to float32's
// precision whatever the inputs' type, and v_mfma_f32_16x16x4_f32 runs at a
// sixteenth of the 16-bit rate. So every float32 operand x is split into two
// halves hi + lo (float16, 11 bits each), after scaling its row or column by
// the power of two that brings its largest element to [2^13, 2^14): an
// element is then held to 22 bits, or to 2^-38 of the largest, and hi.hi +
// hi.lo + lo.hi leaves out 2^-22 of a product. A bfloat16 input is one half
// exactly (to 2^-37 of its row's largest element), so its products with split
// operands take two instructions instead of three. The scales are powers of
// two and leave again in the float32 factor that the result is multiplied with
// anyway. (Two bfloat16 halves would hold 16 bits: 2^-17 of an element.)
//
// The sums inside a matrix instruction are not rounded alike for x and -x: random
// operands come out 1e-9 of the result's size too low on the average, measured,
// which is nothing beside the 5e-8 that they are off by, but all one way. Where q,
// k and v have a mean of their own, sums over thousands of steps gather it: dA and
// ddt_bias were off by 8e-7 and 6e-7. So the backward takes every other of the
// slices, tiles or rows that such a sum goes over with the other sign, in the power
// of two that it is scaled with anyway: 4e-7 and 3e-7.
//
// Layouts of v_mfma_f32_16x16x32_f16, lane l = 16 g + m: A[m][8 g + j],
// B[8 g + j][m] (j = 0..7), D[4 g + i][m] (i = 0..3). The order of the 32
// contraction indices is free as long as A and B agree, so the D of two tiles
// is a B without moving anything between lanes: slot (g, j) stands for row
// 4 g + j of the first tile (j < 4) or 4 g + j - 4 of the second. A wave keeps 16 columns of
// the state for the whole sequence and forms everything that depends on it
// in registers; only K, Q, T and Pm, which all waves share, come through LDS.
#pragma once

#include <hip/hip_runtime.h>

#include "gated_delta.h"

namespace ssm {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr double kLog2eD = 1.4426950408889634;
constexpr int kGdrC = 64;       // steps a chunk
constexpr int kGdrFrags = 6;    // 16 x 32 pieces of a lower triangle of 64: (0,0) (1,0) (2,0) (2,1) (3,0) (3,1)
constexpr int kGdrFragHalves = 64 * 8;

// Index of the piece (row tile tt, half p) among the six.
__device__ __forceinline__ constexpr int gdr_frag(int tt, int p) { return tt < 2 ? tt : 2 * tt - 2 + p; }

__device__ __forceinline__ f32x4_t mfma16(half8_t a, half8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// x, or -x where n is odd.
__device__ __forceinline__ float flip(float x, int n) {
  return __uint_as_float(__float_as_uint(x) ^ (static_cast<uint32_t>(n) << 31));
}

// x, as a value that the compiler cannot trace back: what is computed from it
// inside a loop is not kept in registers across the loop.
__device__ __forceinline__ int anew(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The power of two that brings m >= 0 into [2^13, 2^14), and its inverse.
// m below 2^-100 counts as 2^-100, infinity as 2^127.
struct Pow2 {
  float up, down;
};
__device__ __forceinline__ Pow2 pow2_to_top(float m) {
  uint32_t e = __float_as_uint(m) & 0x7f800000u;  // the exponent where it stands
  e = e > 27u << 23 ? e : 27u << 23;
  e = e < 254u << 23 ? e : 254u << 23;
  return Pow2{__uint_as_float((267u << 23) - e), __uint_as_float(e - (13u << 23))};
}

// Largest value over the lanes l, l ^ 16, l ^ 32, l ^ 48 (those that share a column of D).
__device__ __forceinline__ float col_max(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float w = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(w), __float_as_uint(w), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// Eight scaled values as halves, rounded to nearest even; and what is left of them.
__device__ __forceinline__ half8_t halves(const float (&x)[8]) {
  half8_t h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const half2_t t = __builtin_convertvector((f32x2_t{x[2 * i], x[2 * i + 1]}), half2_t);
    h[2 * i] = t[0];
    h[2 * i + 1] = t[1];
  }
  return h;
}
__device__ __forceinline__ half8_t rest(const float (&x)[8], half8_t h) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i] - static_cast<float>(h[i]);
  return halves(r);
}

// Two D tiles times f as a B operand: its halves and, with LO, what is left.
template <bool LO>
__device__ __forceinline__ void tiles_to_operand(f32x4_t a, f32x4_t b, float f, half8_t& hi, half8_t& lo) {
  const float x[8] = {a[0] * f, a[1] * f, a[2] * f, a[3] * f, b[0] * f, b[1] * f, b[2] * f, b[3] * f};
  hi = halves(x);
  if constexpr (LO) lo = rest(x, hi);
}

template <int T>
__device__ __forceinline__ float tiles_absmax(const f32x4_t (&x)[T]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < T; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(x[j][i]));
  }
  return col_max(m);
}

// Four rows of a column out of a row-major array of halves in LDS: lane m of
// a group of 16 passes the address of row m / 4, columns 4 (m % 4) .. + 3 of a
// 4 x 16 piece, and gets column m.
__device__ __forceinline__ half4_t lds_column4(const _Float16* at) {
  typedef __attribute__((address_space(3))) short4_t* lds_ptr;
  return __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at)));
}

// Eight elements n .. n+7 of row t (rows `step` elements apart from the
// buffer's start), zero past the buffer's end and past `count`. VEC: rows and
// the start on 16-byte boundaries, count a multiple of 8.
template <bool BF16, bool VEC>
struct Raw8 {
  u32x4_t w[BF16 ? 1 : 2];
};
template <bool BF16, bool VEC>
__device__ __forceinline__ Raw8<BF16, VEC> load_raw8(rsrc_t r, int t, int n, uint32_t step, int count) {
  constexpr int EB = BF16 ? 2 : 4;
  Raw8<BF16, VEC> o;
  const uint32_t off = (static_cast<uint32_t>(t) * step + static_cast<uint32_t>(n)) * EB;
  if constexpr (VEC) {
    const uint32_t at = n < count ? off : kOutOfRange;
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
    if constexpr (!BF16) o.w[1] = __builtin_amdgcn_raw_buffer_load_b128(r, n < count ? off + 16 : kOutOfRange, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t at = n + i < count ? off + static_cast<uint32_t>(i * EB) : kOutOfRange;
      if constexpr (BF16) {
        const uint32_t b = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0));
        o.w[0][i / 2] = (i & 1) ? (o.w[0][i / 2] | (b << 16)) : b;
      } else {
        o.w[i / 4][i % 4] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
      }
    }
  }
  return o;
}
template <bool BF16, bool VEC>
__device__ __forceinline__ void raw8_values(const Raw8<BF16, VEC>& o, float (&x)[8]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(o.w[0][i] << 16);
      x[2 * i + 1] = __uint_as_float(o.w[0][i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(o.w[i / 4][i % 4]);
  }
}

// A buffer over `rows` rows of `width` elements, `step` apart.
template <int EB>
__device__ __forceinline__ rsrc_t rows_buffer(const void* base, int64_t at, int rows, uint32_t step, int width) {
  const uint32_t bytes =
      rows > 0 ? (static_cast<uint32_t>(rows - 1) * step + static_cast<uint32_t>(width)) * EB : 0u;
  return raw_buffer(static_cast<const char*>(base) + at * EB, bytes);
}

// What the chunk kernels share of a chunk (an item: (batch row, head, chunk)).
// Per-step factors, 64 floats each:
enum GdrFactor {
  kFacKup = 0,  // power of two that the raw k row is scaled with (backward)
  kFacQup,      // the same for q
  kFacK,        // e^(c_t) |1/k| / kup: row factor of K S
  kFacQ,        // scale e^(c_t) |1/q| / qup: row factor of Q S
  kFacW,        // beta_t e^(c_end - c_t) |1/k| / kup: row factor of E in the state's update
  kFacP,        // 1 / row scale of Pm's halves (backward: Pm^T's)
  kFacEnd,      // [0]: e^(c_end), [1]: 1 / scale of T's halves (one for the whole triangle)
  kFacKn,       // |1/k| / kup (backward)
  kFacQn,       // |1/q| / qup (backward)
  kGdrFactors
};
constexpr int kGdrPieceHalves = kGdrFrags * 2 * kGdrFragHalves;  // T or Pm, hi and lo of every piece

constexpr int kGdrMaxSlots = 32;  // two waves a 16-column slice of a head (P <= 256)
// Largest magnitudes of an item's arrays, one a wave that made a part: the
// scales of the backward's last kernel, which contracts over the columns.
enum GdrMaximum { kMaxS = 0, kMaxE, kMaxX, kMaxDE, kMaxDY, kGdrMaxima };

struct GdrWork {  // device pointers into the workspace
  _Float16* T;    // [items][6][2][64 lanes][8]
  _Float16* Pm;   // the same (forward)
  _Float16* Tt;   // pieces of T^T (backward), order gdr_frag_up
  _Float16* Pt;   // pieces of Pm^T (backward)
  _Float16* K;    // [batch, query/key heads, chunks][1 or 2 halves][64][64 or 128], order kq_at
  _Float16* Q;    // the same
  float* fac;     // [items][kGdrFactors][64]
  float* S;       // [items][P][N] state entering the chunk (backward)
  float* X;       // [items][P][N] gradient of the state leaving it
  float* E;       // [items][64][P]
  float* top;     // [items][kGdrMaxima][kGdrMaxSlots]
  double* part;   // [2][items]: an item's part of dA and of ddt_bias
  float* map;     // [heads][segments][P + N][N]: a segment's map (forward in segments)
  float* seg;     // [segments][heads][P][N]: state entering a segment
  int64_t seg_stride;  // elements from one segment's states to the next's
};

// Pieces of an upper triangle: (0,0) (0,1) (1,0) (1,1) (2,1) (3,1).
__device__ __forceinline__ constexpr int gdr_frag_up(int tt, int p) { return tt < 2 ? 2 * tt + p : tt + 2; }

// Largest |x| over a wave's D tiles, in every lane.
__device__ __forceinline__ float lanes16_max(float v) {
  v = fmaxf(v, quad_xor<1>(v));
  v = fmaxf(v, quad_xor<2>(v));
  v = fmaxf(v, dpp_f<0x141>(v));  // row_half_mirror
  return fmaxf(v, dpp_f<0x140>(v));  // row_mirror
}
__device__ __forceinline__ float lanes16_sum(float v) {
  v += quad_xor<1>(v);
  v += quad_xor<2>(v);
  v += dpp_f<0x141>(v);
  return v + dpp_f<0x140>(v);
}

// Where element n (a multiple of 8, or of 4 for half a slot) of row t of K or
// Q stands among its halves, in LDS and in the workspace alike: rows of NP
// halves without padding, their 16-byte slots exchanged by an exclusive or
// with a number of the row. Both reads of a wave are then free of bank
// conflicts: 16 rows of one slot (an A operand), and four rows of four slots (lds_column4).
template <int NP>
__device__ __forceinline__ int kq_at(int t, int n) {
  const int f = NP == 128 ? ((t & 3) << 2) | ((t >> 2) & 3) : ((t >> 1) & 1) << 2 | ((t >> 2) & 3);
  return t * NP + (((n >> 3) ^ f) << 3) + (n & 7);
}

// The rows of K and Q of a chunk as halves, by a block of 256 threads: four
// lanes a row, 8 elements a piece; into LDS and (keep) into the workspace ([RAW][64]
// [NP] each, lo halves behind the hi ones). kn, qn: a row's norm factor (1
// without the norm) times the inverse of its power of two; kup, qup: that
// power. Rows past `rows` are 0.
template <int NP, bool BF16, bool VEC>
__device__ __forceinline__ void gdr_stage_kq(const GatedDeltaArgs& p, int64_t row0, int rows, int kh, int tid,
                                             _Float16* sK, _Float16* sQ, bool keep, _Float16* gK, _Float16* gQ,
                                             float* kn, float* qn, float* kup, float* qup) {
  constexpr int RAW = BF16 ? 1 : 2;
  const int N = static_cast<int>(p.dstate);
  const int t = tid >> 2, part = tid & 3;
  const rsrc_t rk = rows_buffer<BF16 ? 2 : 4>(p.k, row0 * p.k_step + static_cast<int64_t>(kh) * N, rows,
                                              static_cast<uint32_t>(p.k_step), N);
  const rsrc_t rq = rows_buffer<BF16 ? 2 : 4>(p.q, row0 * p.q_step + static_cast<int64_t>(kh) * N, rows,
                                              static_cast<uint32_t>(p.q_step), N);
  Raw8<BF16, VEC> raw[2][NP / 32];
#pragma unroll
  for (int i = 0; i < NP / 32; ++i) {
    raw[0][i] = load_raw8<BF16, VEC>(rk, t, 32 * i + 8 * part, static_cast<uint32_t>(p.k_step), N);
    raw[1][i] = load_raw8<BF16, VEC>(rq, t, 32 * i + 8 * part, static_cast<uint32_t>(p.q_step), N);
  }
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    float sum = 0.0f, top = 0.0f;
    float x[NP / 32][8];
#pragma unroll
    for (int i = 0; i < NP / 32; ++i) {
      raw8_values<BF16, VEC>(raw[a][i], x[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = fmaf(x[i][e], x[i][e], sum);
        top = fmaxf(top, fabsf(x[i][e]));
      }
    }
    sum += quad_xor<1>(sum);
    sum += quad_xor<2>(sum);
    top = fmaxf(top, quad_xor<1>(top));
    top = fmaxf(top, quad_xor<2>(top));
    const Pow2 s = pow2_to_top(top);
    _Float16 *dst = a == 0 ? sK : sQ, *out = a == 0 ? gK : gQ;
#pragma unroll
    for (int i = 0; i < NP / 32; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= s.up;
      const int at = kq_at<NP>(t, 32 * i + 8 * part);
      const half8_t hi = halves(x[i]);
      *reinterpret_cast<half8_t*>(dst + at) = hi;
      if (keep) *reinterpret_cast<half8_t*>(out + at) = hi;
      if constexpr (RAW == 2) {
        const half8_t lo = rest(x[i], hi);
        *reinterpret_cast<half8_t*>(dst + kGdrC * NP + at) = lo;
        if (keep) *reinterpret_cast<half8_t*>(out + kGdrC * NP + at) = lo;
      }
    }
    if (part == 0) {
      const float n = p.qk_l2norm ? rsqrtf(sum + kL2NormEps) : 1.0f;
      (a == 0 ? kn : qn)[t] = n * s.down;
      (a == 0 ? kup : qup)[t] = s.up;
    }
  }
}

// Inclusive prefix sum over the 64 lanes in double: a chunk's log decays.
__device__ __forceinline__ double wave_prefix(double v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The place of block `block` of a launch among the work's items, so that the
// `group` consecutive items that read the same arrays run on one XCD, whose L2
// then fetches them once: blocks go to the eight XCDs in turn. (Groups are dealt
// one by one, so that rows of different lengths spread; the last groups, where
// there are no eight more, stay in order.)
__device__ __forceinline__ int gdr_xcd_place(int block, int blocks, int group) {
  const int set = 8 * group;
  if (block >= blocks / set * set) return block;
  const int k = block % set;
  return block - k + k % 8 * group + k / 8;
}

// Pairs of waves (16 columns each) a block of the walks over the chunks: as
// many as leave a block for every one of the 256 CUs. Measured (forward of 4096
// steps, bf16, 128 x 128, with 1, 2 and 4 pairs a block): 32 heads 159, 173, 228
// us; 64 heads 353, 247, 285; 128 heads 673, 456, 383.
inline int gdr_block_pairs(int64_t heads, int64_t slices) {
  if (slices >= 4 && heads * ((slices + 3) / 4) >= 256) return 4;
  if (slices >= 2 && heads * ((slices + 1) / 2) >= 256) return 2;
  return 1;
}

// The backward's two walks, forth and back, by one kernel: where a block has one
// pair (few heads: a walk is bound by its own latency, and the two together
// take the time of the longer) and both fit the LDS.
constexpr bool gdr_both_fit(int np, bool bf16) { return np == 64 || bf16; }
inline bool gdr_both_at_once(const GatedDeltaArgs& a) {
  return gdr_both_fit(a.dstate <= 64 ? 64 : 128, a.in_bf16) &&
         gdr_block_pairs(a.batch * a.nheads, (a.headdim + 15) / 16) == 1;
}

// Launchers (0 or a HIP error code). vec: every row of q and k starts on a
// 16-byte boundary and N is a multiple of 8.
int launch_gdr_prep(const GatedDeltaArgs& a, const GdrWork& ws, int64_t chunks, bool backward, bool vec,
                    void* stream);
int launch_gdr_chunk_b(const GatedDeltaArgs& a, const GdrWork& ws, const GdrPlan& pl, bool backward, void* stream);
int launch_gdr_chunk_f(const GatedDeltaArgs& a, const GdrWork& ws, const GdrPlan& pl, bool backward, void* stream);
void launch_gdr_join(const GatedDeltaArgs& a, const GdrWork& ws, int segs, int seg_chunks, hipStream_t st);
int launch_gdr_reverse(const GatedDeltaBwdArgs& a, const GdrWork& ws, int64_t chunks, void* stream);
int launch_gdr_grads(const GatedDeltaBwdArgs& a, const GdrWork& ws, int64_t chunks, void* stream);

}  // namespace ssm
