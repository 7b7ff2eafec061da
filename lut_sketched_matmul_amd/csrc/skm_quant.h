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

__device__ __forceinline__ uint32_t top8(const float* v) {
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu;
    top = top > a ? top : a;
  }
  return top;
}

// Eight values of one lane to eight codes, given the block's exponent byte.
__device__ __forceinline__ u32x2 ckpt_pack8(const float* v, uint32_t s) {
  // 2^-e as fp32: s in [1, 248]; a NaN block (255) stores zeros
  const float r = __builtin_bit_cast(float, (254u - (s == kCkptNaN ? 127u : s)) << 23);
  u32x2 o = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float q = __builtin_rintf(v[j] * r);
    q = __builtin_fminf(__builtin_fmaxf(q, -127.0f), 127.0f);
    const uint32_t c = s == kCkptNaN ? 0u : (uint32_t)(int)q & 0xFFu;
    o[j >> 2] |= c << (8 * (j & 3));
  }
  return o;
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
