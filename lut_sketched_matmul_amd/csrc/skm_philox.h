// Dropout's random numbers: Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel
// random numbers: as easy as 1, 2, 3", 2011), a counter-based generator, so a
// mask is computed again wherever it is needed and never stored.
//
// Value i of a tensor takes half-word i % 8 (low half of word 0 first) of the
// call whose key is seed[0] and whose counter is (i / 8, seed[1]), both as 64
// bits in two words, low word first. It stays when its 16 bits are at least
// round(65536 p): one call serves the eight values that a lane holds in
// one 16-byte load, and p is kept to a multiple of 2^-16.
#pragma once

#include "skm_common.h"

namespace skm {

struct Philox {
  uint32_t k0, k1;  // key
  uint32_t s0, s1;  // upper half of the counter
};

__device__ __forceinline__ Philox philox_of(const int64_t* seed) {
  const uint64_t key = (uint64_t)seed[0], stream = (uint64_t)seed[1];
  return Philox{(uint32_t)key, (uint32_t)(key >> 32), (uint32_t)stream, (uint32_t)(stream >> 32)};
}

__device__ __forceinline__ u32x4 philox_block(const Philox& p, uint64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = p.s0, c3 = p.s1;
  uint32_t k0 = p.k0, k1 = p.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// whether value j (0..7) of a block stays; threshold 65536 keeps none
__device__ __forceinline__ bool philox_stays(u32x4 u, int j, uint32_t threshold) {
  const uint32_t w = u[j >> 1];
  return (j & 1 ? w >> 16 : w & 0xFFFFu) >= threshold;
}

// Two packed 16-bit values (2 j and 2 j + 1 of the block) with those that do not stay cleared
__device__ __forceinline__ uint32_t philox_mask2(u32x4 u, int j, uint32_t threshold, uint32_t v) {
  const uint32_t lo = (u[j] & 0xFFFFu) >= threshold ? v & 0xFFFFu : 0u;
  return lo | ((u[j] >> 16) >= threshold ? v & 0xFFFF0000u : 0u);
}

}  // namespace skm
