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

// (one instruction; from a ^ b ^ c the compiler makes two)
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

__device__ __forceinline__ u32x4 philox_block(const Philox& p, uint64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = p.s0, c3 = p.s1;
  uint32_t k0 = p.k0, k1 = p.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = xor3((uint32_t)(b >> 32), c1, k0);
    c1 = (uint32_t)b;
    c2 = xor3((uint32_t)(a >> 32), c3, k1);
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

// The same for packed 16-bit values, in three packed instructions and an and: those that go are cleared.
struct PhiloxMask {
  uint32_t least;  // the threshold in both halves
  uint32_t all;    // 0 where none stays (a threshold of 65536 has no 16 bits)
};
__device__ __forceinline__ PhiloxMask philox_mask_of(uint32_t threshold) {
  return threshold < 65536u ? PhiloxMask{threshold * 0x00010001u, ~0u} : PhiloxMask{0u, 0u};
}
__device__ __forceinline__ uint32_t philox_mask2(uint32_t u, const PhiloxMask& m, uint32_t v) {
  uint32_t t;
  const uint32_t one = 0x00010001u;
  asm("v_pk_sub_u16 %0, %1, %2 clamp" : "=v"(t) : "s"(m.least), "v"(u));  // 0 where u >= least
  asm("v_pk_min_u16 %0, %1, %2" : "=v"(t) : "v"(t), "s"(one));
  asm("v_pk_sub_u16 %0, %1, %2" : "=v"(t) : "v"(t), "s"(one));            // all bits, or none
  return __builtin_amdgcn_bitop3_b32(t, v, m.all, 0x80);                  // and of the three
}

}  // namespace skm
