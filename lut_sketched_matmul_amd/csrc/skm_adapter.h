// Low-rank adapters of many requests beside a shared projection. Token t has the
// adapter s = ids[t] (none when outside [0, S)), with dropout D in front:
//   h_t  = A_s D(x_t)                       [r]     "down"
//   y_t  = base_t + scale_s B_s h_t         [n]     "up"
//   dh_t = scale_s B_s^T dy_t               [r]     "down" with B's transpose
//   dx_t = base_dx_t + D'(A_s^T dh_t)       [d]     "up" with A's transpose
//   dB_s = sum_t dy_t (scale_s h_t)^T,  dA_s = sum_t dh_t D(x_t)^T      "grad"
// Everything is bound by memory from a few hundred tokens on (r is small beside
// d and n) and by launches and latency below.
//
// Tokens are not sorted for the first four: a tile of 16 or 64 tokens walks the
// distinct adapters among its tokens, multiplies all of its rows by each and
// keeps the rows that are the adapter's. With requests one after the other a
// tile has one or two; in a decode batch of different adapters each adapter's
// weights are read once per tile, which is what they cost in any order. Rows
// never mix: a token is one row of the matrix instruction.
//
// Rounding. Products of 16-bit values are exact and sums fp32. h and dh stay
// fp32; as operands of the matrix cores they are taken as a sum of 16-bit terms:
//   up    two terms (the result is rounded to 16 bits): bf16 16 bits; f16 22 bits
//         of the token's largest |h|, each token scaled by a power of two so
//         that f16's range does not matter
//   grad  three bf16 terms, 24 bits (the gradients are fp32); f16 activations
//         are split into two bf16 terms, which hold all of their bits
// The terms lie side by side along the contraction, so rank 16 with two terms is one
// 32-deep instruction.
#pragma once

#include "skm_launch.h"
#include "skm_philox.h"

namespace skm {
namespace adapt {

constexpr int WAVES = 4;  // of a block
// Over this many tokens the waves of a block take tiles of their own and share the weights through LDS; up to it they
// share a tile and take other columns. Forward calls of both forms (shared / not): 8 adapters of rank 16, 4096 ->
// 11008, 256 tokens 16.0 / 10.7 us, 512 15.7 / 16.0, 1024 22.2 / 25.6; 4 of rank 64, 8192 -> 8192, 256 tokens 20.1 /
// 18.2, 512 22.2 / 27.4, 1024 30.5 / 48.5; one of rank 16, 4096 -> 4096, within 10 % from 64 to 2048 tokens.
constexpr int64_t kManyTokens = 512;
// With many tokens and ranks over this one the waves of "down" share the weights, too (8 adapters of rank 64, 2048
// tokens of 8192 columns: 25 us with the ranges' sum, against 27 to 33); below, a wave keeps its own (4096
// columns, rank 16, 8192 tokens: 18 us against 19 and a sum more).
constexpr int kSharedRank = 32;

template <typename T> __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c);
template <> __device__ __forceinline__ f32x4 mma<half_t>(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x4 mma<bf16_t>(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

constexpr u32x4 kZero4 = {0u, 0u, 0u, 0u};

// Between lanes of one wave that hand values to each other through LDS: what was stored before is there for every lane's
// loads behind it. The hardware completes a wave's LDS operations in order, so this is no instruction; the fences say so
// to the compiler, which may otherwise move a load before a store of another address.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// eight 16-bit values from any address of theirs
template <typename T>
__device__ __forceinline__ u32x4 load_any(const T* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
template <typename T>
__device__ __forceinline__ void store_any(T* p, u32x4 v) {
  __builtin_memcpy(p, &v, 16);
}
// the first `count` (0..8) of them, zeros behind
template <typename T>
__device__ __forceinline__ u32x4 load_some(const T* p, int64_t count) {
  u32x4 v = kZero4;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < count) v[j >> 1] |= (uint32_t)bits16(p[j]) << (16 * (j & 1));
  return v;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)bits16(from_f32<T>(a)) | ((uint32_t)bits16(from_f32<T>(b)) << 16);
}
template <typename T>
__device__ __forceinline__ float unpack(uint32_t w, int half) {
  return to_f32(__builtin_bit_cast(T, (uint16_t)(half ? w >> 16 : w & 0xFFFFu)));
}

// Eight fp32 values as two terms of T: rounded, and what that takes away rounded (zero beside a term that is not
// finite)
template <typename T>
__device__ __forceinline__ void split8(const float (&v)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = v[2 * j], b = v[2 * j + 1];
    hi[j] = pack2<T>(a, b);
    const float c = unpack<T>(hi[j], 0), d = unpack<T>(hi[j], 1);
    lo[j] = pack2<T>(__builtin_isfinite(c) ? a - c : 0.f, __builtin_isfinite(d) ? b - d : 0.f);
  }
}

// Rows e = 0..7 of eight values each, turned: out[e] holds value e of every row
__device__ __forceinline__ void turn8x8(const u32x4 (&row)[8], u32x4 (&out)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      out[e][j] = __builtin_amdgcn_perm(row[2 * j + 1][e >> 1], row[2 * j][e >> 1],
                                        e & 1 ? 0x07060302u : 0x05040100u);
}

// The adapters of a tile of up to 64 tokens, one token a lane: walks them, each
// with the lanes that have it. The same in every wave of a block.
struct TileIds {
  int id;          // this lane's token's adapter, -1 = none
  uint64_t left;   // lanes not walked yet
  __device__ __forceinline__ TileIds(const int32_t* ids, int S, int64_t t, bool in) {
    id = !in ? -1 : (ids ? ids[t] : 0);
    if (id >= S || id < 0) id = -1;
    left = __ballot(id >= 0);
  }
  __device__ __forceinline__ bool next(int& a, uint64_t& lanes) {
    if (!left) return false;
    a = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(left));
    lanes = __ballot(id == a);
    left &= ~lanes;
    return true;
  }
};

// "down": parts[split][t][rp] = the split's range of the contraction of P [m][K] with
// row-major W [S][rows r at ldw]; P's rows start at 16 bytes when K % 8 == 0
struct Down {
  const void* P;
  const void* W;
  int64_t ldw, wstride;  // between W's rows and adapters, in elements
  int64_t m, K, per;     // per: contraction of one split, a multiple of 64
  int r, rp, S, splits;
  const int32_t* ids;
  Dropout drop;  // of P (threshold 0 = none)
  float* parts;
};
int down_splits(int64_t m, int64_t K, int r, int S, int64_t& per);
// (a.splits is what is left for the reader to add up)
hipError_t launch_down(Down& a, int dtype, hipStream_t s);

// "up": out [m][N] = base + sum over ranks of factor_t h_t[k] W[column][k], h_t the sum of
// `splits` parts; forward: W = B, base and out of T; backward: W = A, base fp32, dropout
struct Up {
  const float* parts;
  int splits, rp, r, S;
  const void* W;
  int64_t m, N;
  const int32_t* ids;
  const float* scale;  // factor of the adapter, NULL = 1
  float factor;        // and of all
  const void* base;    // NULL = zeros
  void* out;
  float* H;  // forward: [m][r] the sums of the parts, NULL = not wanted
  Dropout drop;
};
hipError_t launch_up(const Up& a, int dtype, bool back, hipStream_t s);

// the whole forward of a few tokens in one launch, without a workspace
bool few_tokens(const AdapterArgs& a);
hipError_t launch_few(const AdapterArgs& a, const void* base, void* Y, float* H, hipStream_t s);

// ranks padded to whole groups of eight in the parts
inline int padded_rank(int r) { return (r + 7) / 8 * 8; }

}  // namespace adapt
}  // namespace skm
