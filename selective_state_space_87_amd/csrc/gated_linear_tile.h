// Tiles of the gated linear recurrence (gfx950): 64 channels and a number of
// steps, a block of 256 threads each, and the chain that joins the tiles of a
// channel.
//
// A thread has VC adjacent channels (forward one 16-byte load of x or a gate, 8 of
// bfloat16 or 4 of float32; backward 4, whose float32 gradients are 16 bytes; at
// whatever boundary the row starts on), and some consecutive steps, a slice:
// consecutive lanes have consecutive channels, so a load of a wave reads whole rows
// of the tile. All a tile's loads are issued before the first is used.
//
// A recurrence h <- a h + b over some steps is the map h -> P h + S (P the product
// of the a, S the result from 0), and maps join as (P2 P1, P2 S1 + S2). In the
// tile slices are joined through LDS: 256 threads as 64 channels of 4 runs of
// slices. Over the tiles there is the chain: every tile publishes its map, and
// one in kGlrWindow the state behind it; a tile reads the last such state
// before it and the maps from there on, all at once, and joins them in order.
// So the input is read once, the joins are the same in every run (results are
// deterministic), and the serial part is one exchange through memory every
// kGlrWindow tiles. (Reading it twice, for the maps and for the states, would
// take 14 bytes an element for 8.) Where P underflows to 0, a finite state loses less than
// 2^-149 of itself; an infinite one becomes NaN, where step by step it stays infinite.
// (Telling such a P from a decay of 0 would take instructions an element.)
//
// Waiting always ends. A block takes its tile by a ticket (an atomic count of its
// group's), and tickets go along the chain: what a tile waits for is held by a block that
// started earlier, which publishes its map before it waits, and its state after
// waiting for earlier ones only; the first waits for nothing. A wait also
// ends by itself, with NaN, after kGlrMostPolls tries (some 0.4 s, where 10 us are
// usual), should two calls at once have been given the same workspace; a block
// whose ticket, then, is past the last tile does nothing.
//
// Data travel in the words themselves (64 bits: the map or the state and a mark),
// so no fence is needed: a word is either not there (all ones, as cleared
// before the launch) or whole.
#pragma once

#include <hip/hip_runtime.h>

#include "gated_linear.h"

namespace ssm {

constexpr int kGlrThreads = 256;
constexpr int kGlrRuns = kGlrThreads / kGlrChannels;  // runs of slices
constexpr uint32_t kGlrMissing = 0xffffffffu;
constexpr int kGlrMostPolls = 1 << 18;

// ---- a thread's inputs of one step

// How 256 threads lie on a tile of STEPS steps, with VC channels a thread.
template <int VC, int STEPS>
struct GlrShape {
  static constexpr int kLanes = kGlrChannels / VC;        // threads over the channels
  static constexpr int kSlices = kGlrThreads / kLanes;    // slices of a tile
  static constexpr int kSteps = STEPS / kSlices;          // steps of a slice
  static constexpr int kRun = kSlices / kGlrRuns;         // slices of a run
};

// VC elements in as many words as they take; any element boundary (the memory
// unit takes all), read once: past the caches.
template <bool BF16, int VC>
struct GlrPack {
  static constexpr int N = BF16 ? VC / 2 : VC;
  typedef uint32_t Words __attribute__((ext_vector_type(N)));
  typedef uint32_t Any __attribute__((ext_vector_type(N), aligned(BF16 ? 2 : 4)));
};

// Elements at .. at + VC - 1, of which `left` are there (zeros for the others).
template <bool BF16, int VC, bool ONCE = true>
__device__ __forceinline__ typename GlrPack<BF16, VC>::Words glr_load(const void* base, int64_t at, int left) {
  using Pack = GlrPack<BF16, VC>;
  typename Pack::Words w = {};
  if (left >= VC) {
    const auto* from = reinterpret_cast<const typename Pack::Any*>(static_cast<const char*>(base) + at * (BF16 ? 2 : 4));
    if constexpr (ONCE) {
      w = __builtin_nontemporal_load(from);
    } else {
      w = *from;
    }
  } else {
#pragma unroll
    for (int c = 0; c < VC; ++c) {
      if (c < left) {
        const uint32_t e = load_bits<BF16>(base, at + c);
        if constexpr (BF16) {
          w[c / 2] |= e << (16 * (c & 1));
        } else {
          w[c] = e;
        }
      }
    }
  }
  return w;
}

template <bool BF16, typename W>
__device__ __forceinline__ float glr_elem(const W& w, int c) {
  if constexpr (BF16) {
    return __uint_as_float(c & 1 ? w[c / 2] & 0xffff0000u : w[c / 2] << 16);
  } else {
    return __uint_as_float(w[c]);
  }
}

// float32 parameters and states: several blocks read the same.
template <int VC>
__device__ __forceinline__ void glr_load_f32(const float* base, int64_t at, int left, float (&v)[VC]) {
#pragma unroll
  for (int q = 0; q < VC / 4; ++q) {
    const auto w = glr_load<false, 4, false>(base, at + 4 * q, left - 4 * q);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[4 * q + c] = __uint_as_float(w[c]);
  }
}

template <bool BF16, int VC>
__device__ __forceinline__ void glr_store(void* base, int64_t at, int left, const float (&v)[VC]) {
  using Pack = GlrPack<BF16, VC>;
  if (left >= VC) {
    typename Pack::Any w;
#pragma unroll
    for (int i = 0; i < Pack::N; ++i) {
      if constexpr (BF16) {
        w[i] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i])) |
               (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i + 1])) << 16);
      } else {
        w[i] = __float_as_uint(v[i]);
      }
    }
    __builtin_nontemporal_store(w, reinterpret_cast<typename Pack::Any*>(static_cast<char*>(base) + at * (BF16 ? 2 : 4)));
  } else {
#pragma unroll
    for (int c = 0; c < VC; ++c) {
      if (c < left) store_elem<BF16>(base, at + c, v[c]);
    }
  }
}

// Inputs of a thread's slice, TS steps from tile step `s0` on, n steps of the
// tile being there. A tile that is there whole is loaded without a branch, so
// that all loads are on their way before the first is waited for.
template <bool BF16, bool GATED, int VC, int TS>
struct GlrRaw {
  typename GlrPack<BF16, VC>::Words x[TS], gate[TS], igate[GATED ? TS : 1];

  // Hides from the compiler that the gates' words are those it has seen, so that what was
  // made of them is made again from here on, not kept: in the backward that would take 177
  // registers, where three blocks a CU leave 168 (training step (8, 2048, 1536) 184 us
  // for 170).
  template <int ACT>
  __device__ __forceinline__ void forget() {
    const auto hide = [](auto& words) __attribute__((always_inline)) {
#pragma unroll
      for (int w = 0; w < GlrPack<BF16, VC>::N; ++w) {
        uint32_t bits = words[w];
        asm volatile("" : "+v"(bits));
        words[w] = bits;
      }
    };
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      if constexpr (ACT != kGateRaw) hide(gate[i]);
      if constexpr (GATED) hide(igate[i]);
    }
  }

  __device__ __forceinline__ void load(const GatedLinearArgs& p, int64_t row, int c, int left, int s0, int n, bool whole) {
    const int64_t ax = (row + s0) * p.x_step + c, ag = (row + s0) * p.gate_step + c;
    const int64_t ai = GATED ? (row + s0) * p.igate_step + c : 0;
    if (whole) {
#pragma unroll
      for (int i = 0; i < TS; ++i) {
        gate[i] = glr_load<BF16, VC>(p.gate, ag + i * p.gate_step, VC);
        x[i] = glr_load<BF16, VC>(p.x, ax + i * p.x_step, VC);
        if constexpr (GATED) igate[i] = glr_load<BF16, VC>(p.igate, ai + i * p.igate_step, VC);
      }
    } else {
#pragma unroll
      for (int i = 0; i < TS; ++i) {
        const int have = s0 + i < n ? left : 0;
        gate[i] = glr_load<BF16, VC>(p.gate, ag + i * p.gate_step, have);
        x[i] = glr_load<BF16, VC>(p.x, ax + i * p.x_step, have);
        if constexpr (GATED) igate[i] = glr_load<BF16, VC>(p.igate, ai + i * p.igate_step, have);
      }
    }
  }
};

// A thread's channels' parameters, scaled as gated_linear.h takes them.
template <int VC, int ACT, bool GATED>
struct GlrParams {
  float A2[VC], gbias[VC], ibias[VC];

  __device__ __forceinline__ void load(const GatedLinearArgs& p, int c, int left) {
    glr_load_f32<VC>(p.A, c, left, A2);
#pragma unroll
    for (int v = 0; v < VC; ++v) A2[v] *= kLog2e, gbias[v] = ibias[v] = 0.0f;
    if (p.gbias != nullptr) glr_load_f32<VC>(p.gbias, c, left, gbias);
    if (GATED && p.ibias != nullptr) glr_load_f32<VC>(p.ibias, c, left, ibias);
  }
};

// Decays a and inputs b of a slice. (Steps that are not there: see glr_mask.) Four
// channels at a time, in the order in which the loads come: scheduled over the whole
// slice all loads are waited for first, and some forms spill ((4, 8192, 4096) bfloat16 227
// us for 212).
template <bool BF16, int ACT, int SCALE, bool GATED, int TS, int VC>
__device__ __forceinline__ void glr_elements(const GlrRaw<BF16, GATED, VC, TS>& raw, const GlrParams<VC, ACT, GATED>& par,
                                             float (&a)[TS][VC], float (&b)[TS][VC]) {
#pragma unroll
  for (int i = 0; i < TS; ++i) {
#pragma unroll
    for (int v = 0; v < VC; ++v) {
      const float t = par.A2[v] * gate_value<ACT>(glr_elem<BF16>(raw.gate[i], v) + par.gbias[v]);
      a[i][v] = exp2_hw(t);
      b[i][v] = glr_elem<BF16>(raw.x[i], v) * input_weight<SCALE>(t, a[i][v]);
      if constexpr (GATED) b[i][v] *= glr_sigmoid(glr_elem<BF16>(raw.igate[i], v) + par.ibias[v]);
      if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Steps from the n-th of the tile on leave the state: decay 1, input 0.
template <int TS, int VC>
__device__ __forceinline__ void glr_mask(int s0, int n, float (&a)[TS][VC], float (&b)[TS][VC]) {
#pragma unroll
  for (int i = 0; i < TS; ++i) {
    const bool on = s0 + i < n;
#pragma unroll
    for (int v = 0; v < VC; ++v) a[i][v] = on ? a[i][v] : 1.0f, b[i][v] = on ? b[i][v] : 0.0f;
  }
}

// ---- the place of a group, 64 channels of a batch row

struct GlrGroup {
  int64_t row0;   // first row of its batch row in [B L, ..]
  int64_t steps;  // steps that the batch row has
  int b, c0;      // batch row, first channel
};

__device__ __forceinline__ GlrGroup glr_group(const GatedLinearArgs& p, uint32_t group) {
  GlrGroup t;
  const uint32_t per_row = static_cast<uint32_t>((p.dim + kGlrChannels - 1) / kGlrChannels);
  t.b = static_cast<int>(group / per_row);
  t.c0 = static_cast<int>(group % per_row) * kGlrChannels;
  t.row0 = static_cast<int64_t>(t.b) * p.seqlen;
  t.steps = gdr_row_steps(p.seqlens, t.b, p.seqlen);
  return t;
}

// ---- the chain

struct GlrChain {
  uint32_t* tickets;  // a count a group, kGlrTicketBytes apart
  uint64_t* maps;     // [tile][group][64]: S, and P (never all ones) above
  uint64_t* states;   // [window][group][64]: the state, and 0 above
  uint32_t groups, columns, tiles;
};

inline GlrChain glr_chain(const GlrChainPlan& p, void* workspace) {
  char* w = static_cast<char*>(workspace);
  return GlrChain{reinterpret_cast<uint32_t*>(w), reinterpret_cast<uint64_t*>(w + p.off_words),
                  reinterpret_cast<uint64_t*>(w + p.off_states), static_cast<uint32_t>(p.groups),
                  static_cast<uint32_t>(p.columns), static_cast<uint32_t>(p.tiles)};
}

__device__ __forceinline__ uint64_t glr_word(float low, uint32_t high) {
  return static_cast<uint64_t>(__float_as_uint(low)) | (static_cast<uint64_t>(high) << 32);
}
__device__ __forceinline__ void glr_put(uint64_t* at, uint64_t w) {
  __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t glr_get(const uint64_t* at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One wave: the state that enters place `q` of the chain, given the map (P, S) of
// the tile there and the state `start` that enters place 0. Lane l has channel l.
__device__ __forceinline__ float glr_enter(const GlrChain& c, uint32_t group, uint32_t q, float P, float S, float start) {
  const int lane = threadIdx.x % kGlrChannels;
  const auto at = [&](uint32_t place) {
    return (static_cast<int64_t>(place) * c.groups + group) * kGlrChannels + lane;
  };
  uint32_t high = __float_as_uint(P);
  if (high == kGlrMissing) high = 0x7fc00000u;  // one NaN for another
  // h_final may be h0: the start has been read before the last tile, which waits for this map, can write it.
  asm volatile("" : : "v"(start) : "memory");
  glr_put(c.maps + at(q), glr_word(S, high));
  const uint32_t window = q / kGlrWindow, j = q % kGlrWindow;
  // All words are read at once, with no branch between (each read takes 1 us or more
  // through the memory that the XCDs share): those that are not needed are this
  // place's own.
  const uint64_t* from[kGlrWindow];
#pragma unroll
  for (uint32_t i = 0; i < kGlrWindow - 1; ++i) from[i] = c.maps + at(i < j ? q - j + i : q);
  from[kGlrWindow - 1] = window > 0 ? c.states + at(window - 1) : c.maps + at(q);
  uint64_t word[kGlrWindow];
  for (int tries = 0;; ++tries) {
#pragma unroll
    for (uint32_t i = 0; i < kGlrWindow; ++i) word[i] = glr_get(from[i]);
    bool missing = false;
#pragma unroll
    for (uint32_t i = 0; i < kGlrWindow; ++i) missing |= static_cast<uint32_t>(word[i] >> 32) == kGlrMissing;
    if (!__any(missing)) break;
    if (tries == kGlrMostPolls) {
      start = __uint_as_float(0x7fc00000u);
      word[kGlrWindow - 1] = glr_word(start, 0);
      break;
    }
    __builtin_amdgcn_s_sleep(1);
  }
  float h = window > 0 ? __uint_as_float(static_cast<uint32_t>(word[kGlrWindow - 1])) : start;
#pragma unroll
  for (uint32_t i = 0; i < kGlrWindow - 1; ++i) {
    const float P0 = __uint_as_float(static_cast<uint32_t>(word[i] >> 32)), S0 = __uint_as_float(static_cast<uint32_t>(word[i]));
    h = i < j ? fmaf(P0, h, S0) : h;
  }
  if (j == kGlrWindow - 1) glr_put(c.states + at(window), glr_word(fmaf(P, h, S), 0));
  return h;
}

// The block's tile of its group's chain, or kGlrNoTile for a block of no group.
// Blocks of one group are `columns` apart, a multiple of 8, so that they run on one
// XCD and neighbouring channels on the same: rows are read in pieces of some KB
// (with neighbours on different XCDs (4, 8192, 4096) took 257 us in place of 239). A count
// a group: one for all would be the bound, 12 ns a tile (33000 tiles 420 us).
template <bool BACK>
__device__ __forceinline__ uint32_t glr_ticket(const GlrChain& c, uint32_t* slot, uint32_t* group) {
  *group = blockIdx.x % 8 * (c.columns / 8) + blockIdx.x / 8 % (c.columns / 8);
  if (*group >= c.groups) return kGlrNoTile;
  if (threadIdx.x == 0) *slot = atomicAdd(c.tickets + *group * (kGlrTicketBytes / 4), 1u);
  __syncthreads();
  return glr_tile_of(*slot, c.tiles, BACK);
}

// Clears a chain's words to "not there" and its count to 0 (a kernel, not a memset: graphs take it).
void launch_glr_clear(const GlrChainPlan& p, void* workspace, hipStream_t st);

// f(act, scale, with an input gate) as compile-time constants.
template <typename F>
void glr_by_form(const GatedLinearArgs& p, F&& f) {
  using std::integral_constant;
  const auto gated = [&](auto act, auto scale) {
    p.igate != nullptr ? f(act, scale, std::true_type{}) : f(act, scale, std::false_type{});
  };
  const auto scale = [&](auto act) {
    if (p.scale == kInputNorm) {
      gated(act, integral_constant<int, kInputNorm>{});
    } else if (p.scale == kInputComplement) {
      gated(act, integral_constant<int, kInputComplement>{});
    } else {
      gated(act, integral_constant<int, kInputPlain>{});
    }
  };
  if (p.act == kGateSigmoid) {
    scale(integral_constant<int, kGateSigmoid>{});
  } else if (p.act == kGateSoftplus) {
    scale(integral_constant<int, kGateSoftplus>{});
  } else {
    scale(integral_constant<int, kGateRaw>{});
  }
}

template <bool BF16>
void launch_glr_fwd(const GatedLinearArgs& a, const GlrChainPlan& plan, hipStream_t st);
template <bool BF16>
void launch_glr_bwd(const GatedLinearBwdArgs& a, const GlrBwdPlan& plan, hipStream_t st);

}  // namespace ssm
