// The 8-bit checkpoint of an activation row: int8 codes q and one exponent
// byte s per block of 32 columns, value q 2^(s - 127).
//
// e = s - 127 is the smallest integer with 127 2^e >= M, M the block's largest
// magnitude, clamped so that every value q 2^e is a finite number of the
// activations' type that the type holds exactly: [-24, 9] for f16 (its
// subnormals are multiples of 2^-24; 127 2^9 = 65024), [-126, 121] for bf16
// and fp32. q = x 2^-e rounded to nearest even (the product is exact),
// clamped to [-127, 127]: off by at most half a step, and by less than one
// where the upper clamp applies (M > 127 2^9, or 127 2^121). A power of two
// as the scale keeps q 2^e exact in bf16 (7 significant bits), so matrix
// products read the checkpoint without another rounding. A block that holds
// an infinity or a NaN is stored as s = 255, q = 0 and reads back as NaN.
#pragma once

#include "skm_common.h"

namespace skm {

constexpr int kCkptBlock = 32;          // columns per exponent byte
constexpr uint32_t kCkptNaN = 255u;     // exponent byte of a block with a non-finite value

template <typename T> struct ckpt_range { static constexpr int lo = -126, hi = 121; };
template <> struct ckpt_range<half_t> { static constexpr int lo = -24, hi = 9; };

// exponent byte from the bit pattern of the block's largest magnitude (fp32)
template <typename T>
__device__ __forceinline__ uint32_t ckpt_exp_of(uint32_t top) {
  if (top >= 0x7F800000u) return kCkptNaN;
  // top = f 2^k: 127 2^e >= top at e = k - 6 when f <= 127 / 64, else at k - 5
  int e = (int)(top >> 23) - 127 - 6 + ((top & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  e = e < ckpt_range<T>::lo ? ckpt_range<T>::lo : (e > ckpt_range<T>::hi ? ckpt_range<T>::hi : e);
  return (uint32_t)(e + 127);
}

// largest bit pattern over the four lanes of a quad (one block: 8 columns per lane)
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
  return v > o ? v : o;
}

// Largest magnitude of eight values as an fp32 bit pattern (NaN above
// infinity): of fp32 values, or of 16-bit ones packed as stored, whose patterns
// without the sign order like their magnitudes (four packed maxima).
__device__ __forceinline__ uint32_t top8(const float* v) {
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu;
    top = top > a ? top : a;
  }
  return top;
}
__device__ __forceinline__ uint32_t top8_16(u32x4 w) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = __builtin_bit_cast(u16x2, w[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int q = 1; q < 4; ++q) {
    const uint32_t a = w[q] & 0x7FFF7FFFu;
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, a));
  }
  return m.x > m.y ? m.x : m.y;
}
template <typename T> __device__ __forceinline__ uint32_t f32_bits_of(uint32_t p) {
  return __builtin_bit_cast(uint32_t, to_f32(__builtin_bit_cast(T, (uint16_t)p)));
}

// Eight values of one lane to eight codes, given the block's exponent byte.
// x 2^-e + 1.5 2^23 rounds x 2^-e to an integer (nearest even, the product is
// exact) and holds it in its low byte.
__device__ __forceinline__ u32x2 ckpt_pack8(const float* v, uint32_t s) {
  // 2^-e as fp32: s in [1, 248]; a NaN block (255) stores zeros
  const bool ok = s != kCkptNaN;
  const float r = __builtin_bit_cast(float, (254u - (ok ? s : 127u)) << 23);
  constexpr float M = 12582912.0f;
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    c[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(__builtin_fmaf(v[j], r, M), M - 127.0f, M + 127.0f));
  u32x2 o;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t a = __builtin_amdgcn_perm(c[4 * q + 1], c[4 * q], 0x0C0C0400u);
    const uint32_t b = __builtin_amdgcn_perm(c[4 * q + 3], c[4 * q + 2], 0x0C0C0400u);
    o[q] = ok ? a | b << 16 : 0u;
  }
  return o;
}

// The checkpoint of eight values as stored in T (`w`, 16 or 32 bytes), one
// lane's part of its block: codes, and the block's exponent byte in `s`.
template <typename T>
__device__ __forceinline__ u32x2 ckpt_of(const u32x4* w, uint32_t& s) {
  float v[8];
  if constexpr (__is_same(T, float)) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      // (the vector as a whole: see mm::ld_f4)
      const f32x4 a = __builtin_bit_cast(f32x4, w[q]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * q + j] = a[j];
    }
    s = ckpt_exp_of<T>(quad_max(top8(v)));
  } else {
    s = ckpt_exp_of<T>(f32_bits_of<T>(quad_max(top8_16(w[0]))));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t p = w[0][j >> 1];
      v[j] = to_f32(__builtin_bit_cast(T, (uint16_t)(j & 1 ? p >> 16 : p & 0xFFFFu)));
    }
  }
  return ckpt_pack8(v, s);
}

// Eight codes back to values (fp32, exact).
__device__ __forceinline__ void ckpt_unpack8(u32x2 c, uint32_t s, float* v) {
  const float step = s == kCkptNaN ? __builtin_nanf("") : __builtin_bit_cast(float, s << 23);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)(int)(int8_t)(c[j >> 2] >> (8 * (j & 3))) * step;
}

// Eight consecutive values p[0..7] (16-byte aligned) to fp32, and back with
// rounding to nearest even.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  if constexpr (__is_same(T, float)) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = to_f32(__builtin_bit_cast(T, (uint16_t)(a[j] & 0xFFFFu)));
      v[2 * j + 1] = to_f32(__builtin_bit_cast(T, (uint16_t)(a[j] >> 16)));
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v) {
  if constexpr (__is_same(T, float)) {
    reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = (uint32_t)bits16(from_f32<T>(v[2 * j])) | ((uint32_t)bits16(from_f32<T>(v[2 * j + 1])) << 16);
    *reinterpret_cast<u32x4*>(p) = o;
  }
}

}  // namespace skm
