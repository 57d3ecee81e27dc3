// Random bits of the dropout: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011). A block of eight
// consecutive elements takes the four words at counter (block's low and high
// word, step, call) under the 64-bit key `seed`: element e the (e mod 8)-th
// half word, low half first. Sixteen bits an element: the ten rounds (some 110
// instructions, 20 of them products at a quarter of the rate) take 21 issue slots an
// element so, where a bfloat16 array's 4 bytes take 30 slots' time to cross HBM; with
// 32 bits they would serve four elements and take 42.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

struct DropKey {
  uint32_t k0, k1, step, call;
  uint32_t threshold;  // an element is kept where its 16 bits are at least this (0 .. 65536)
  float scale;         // 65536 / (65536 - threshold)
};

__device__ __forceinline__ DropKey drop_key(const int64_t* rng, uint32_t call, uint32_t threshold, float scale) {
  const uint64_t seed = static_cast<uint64_t>(rng[0]);
  return DropKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(rng[1]), call,
                 threshold, scale};
}

__device__ __forceinline__ void drop_words(const DropKey& k, uint64_t block, uint32_t* w) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32), c2 = k.step, c3 = k.call;
  uint32_t k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

// Eight consecutive elements from element e on: kept and scaled, or zero. (The
// product is rounded by itself, so that every kernel gives the same value,
// whatever it adds next.)
__device__ __forceinline__ void drop8(const DropKey& k, uint64_t e, float (&v)[8]) {
#pragma clang fp contract(off)
  uint32_t w[8];
  const int s = static_cast<int>(e & 7);
  drop_words(k, e >> 3, w);
  if (s != 0) {  // rows of widths that are not multiples of eight: the half words s .. s + 7 of two blocks
    drop_words(k, (e >> 3) + 1, w + 4);
    if (s & 4) {
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (s & 2) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (s & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_alignbit(w[i + 1], w[i], 16);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (w[i] & 0xffffu) >= k.threshold ? v[2 * i] * k.scale : 0.0f;
    v[2 * i + 1] = (w[i] >> 16) >= k.threshold ? v[2 * i + 1] * k.scale : 0.0f;
  }
}

}  // namespace ssm
