// Epilogues of the forward tiles (skm_gemm_fwd.h) for the cross entropy: see
// skm_xent.h for the mathematics.
#pragma once

#include "skm_gemm_fwd.h"
#include "skm_xent.h"

namespace skm {

namespace {

struct XentRows {
  const int32_t* rows;   // [count] token of each listed row
  const int32_t* count;
  const int64_t* targets;  // [m]
  int64_t v0;              // first vocabulary row of the launch
};

// (target - first column of the lane's outputs) or -1, for a lane's token:
// its outputs are columns c0 + 32 jj + 8 q + 4 (lane / 32) + 0..3
__device__ __forceinline__ int target_in_wave(int64_t target, int64_t c0, int lane) {
  const int64_t r = target - c0;
  return r >= 0 && r < 64 ? (int)r - 4 * (lane >> 5) : -64;
}

static_assert(G_BN == 256, "the statistics are laid out per 256 words");

// EpStats: part[(n0 / 256) * stride + c] = (max, sum of exp(z - max)) over the
// block's columns for listed token c; tlogit[c] = the target's logit (written
// by the one lane that holds it).
template <typename TX> struct EpStats {
  static constexpr bool SWAP = true, ROWS = true;
  struct Args : XentRows {
    float2* part;
    int64_t stride;
    float* tlogit;
  };
  template <bool SC>
  static __device__ __forceinline__ void run(const f32x16 (&acc)[4][2], const Args& ep,
                                             const int32_t* __restrict__ rexp, int64_t m, int64_t n, int64_t m0,
                                             int64_t n0, int wm, int wn, int lane, int t) {
    const int64_t c0 = n0 + 64 * wn;
    const int cols = (int)(n - c0 < 64 ? n - c0 : 64) - 4 * (lane >> 5);  // valid columns from the lane's first
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 128 * wm + 32 * i + (lane & 31);
      const int64_t tok = m0 + row;
      const int64_t src = ep.rows[tok < m ? tok : m - 1];
      const float u = SC ? pow2f(rexp[src]) : 1.0f;
      const int tgt = target_in_wave(ep.targets[src], ep.v0 + c0, lane);
      float mx = -__builtin_inff();
      float tl = 0.0f;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int col = 32 * jj + 8 * (e >> 2) + (e & 3);
          const float z = SC ? acc[i][jj][e] * u : acc[i][jj][e];
          if (col < cols) mx = __builtin_fmaxf(mx, z);
          if (col == tgt) tl = z;
        }
      if (tgt >= 0 && (tgt & 4) == 0 && tok < m) ep.tlogit[tok] = tl;
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float ref = mx == -__builtin_inff() ? 0.0f : mx;
      float sum = 0.0f;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int col = 32 * jj + 8 * (e >> 2) + (e & 3);
          const float z = SC ? acc[i][jj][e] * u : acc[i][jj][e];
          sum += col < cols ? __expf(z - ref) : 0.0f;
        }
      sum += __shfl_xor(sum, 32, 64);
      if (lane < 32) {
        mm::st_w((uint32_t)(wn * G_BM + row) * 8u, __builtin_bit_cast(uint32_t, mx));
        mm::st_w((uint32_t)(wn * G_BM + row) * 8u + 4u, __builtin_bit_cast(uint32_t, sum));
      }
    }
    __syncthreads();
    if (t < G_BM && m0 + t < m) {
      float a[4], b[4];
      float mx = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        a[w] = __builtin_bit_cast(float, mm::ld_w((uint32_t)(w * G_BM + t) * 8u));
        b[w] = __builtin_bit_cast(float, mm::ld_w((uint32_t)(w * G_BM + t) * 8u + 4u));
        mx = __builtin_fmaxf(mx, a[w]);
      }
      const float ref = mx == -__builtin_inff() ? 0.0f : mx;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) sum += b[w] * __expf(a[w] - ref);
      ep.part[n0 / G_BN * ep.stride + m0 + t] = float2{mx, sum};
    }
  }
};

// EpGrad: dZ of the block, [listed token][ld] in up to three forms (NULL =
// not wanted): hi + lo in TX for dLUT (hi also for dX when the tables have
// that dtype) and dxv in TL for dX. Columns n .. ld - 1 and listed rows past
// the count up to the next multiple of 32 are written as zeros.
template <typename TX, typename TL> struct EpGrad {
  static constexpr bool SWAP = true, ROWS = true;
  struct Args : XentRows {
    const float* lse;    // [m]
    const float* dloss;  // [m]
    const float* scale;
    int64_t V, ld;
    TX* hi;
    TX* lo;
    TL* dxv;
  };
  template <bool SC>
  static __device__ __forceinline__ void run(const f32x16 (&acc)[4][2], const Args& ep,
                                             const int32_t* __restrict__ rexp, int64_t m, int64_t n, int64_t m0,
                                             int64_t n0, int wm, int wn, int lane, int t) {
    const int64_t c0 = n0 + 64 * wn;
    const int64_t mpad = (m + 31) / 32 * 32;
    const int cols = (int)(n - c0 < 64 ? n - c0 : 64) - 4 * (lane >> 5);
    const int stored = (int)(ep.ld - c0 < 64 ? ep.ld - c0 : 64) - 4 * (lane >> 5);
    const float scale = *ep.scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t tok = m0 + 128 * wm + 32 * i + (lane & 31);
      if (tok >= mpad) continue;
      const bool live = tok < m;
      const int64_t src = ep.rows[live ? tok : m - 1];
      const float u = SC ? pow2f(rexp[src]) : 1.0f;
      const int64_t target = ep.targets[src];
      const int tgt = target_in_wave(target, ep.v0 + c0, lane);
      const float lse = ep.lse[src];
      // a target outside the vocabulary gives NaN gradients (its loss is NaN)
      const float gs = target >= 0 && target < ep.V ? ep.dloss[src] * scale : __builtin_nanf("");
      const int64_t at = tok * ep.ld + c0 + 4 * (lane >> 5);
#pragma unroll
      for (int jj = 0; jj < 2; ++jj)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int cq = 32 * jj + 8 * q;
          if (cq >= stored) continue;
          float g[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float z = SC ? acc[i][jj][4 * q + k] * u : acc[i][jj][4 * q + k];
            const float p = __expf(z - lse) - (cq + k == tgt ? 1.0f : 0.0f);
            g[k] = live && cq + k < cols ? p * gs : 0.0f;
          }
          if (ep.hi) {
            uint32_t h[2] = {mm::pack_tc<TX>(g[0], g[1]), mm::pack_tc<TX>(g[2], g[3])};
            *reinterpret_cast<u32x2*>(ep.hi + at + cq) = u32x2{h[0], h[1]};
            if (ep.lo) {
              float r[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                r[k] = g[k] - to_f32(__builtin_bit_cast(TX, (uint16_t)(h[k >> 1] >> (16 * (k & 1)))));
              *reinterpret_cast<u32x2*>(ep.lo + at + cq) =
                  u32x2{mm::pack_tc<TX>(r[0], r[1]), mm::pack_tc<TX>(r[2], r[3])};
            }
          }
          if (ep.dxv)
            *reinterpret_cast<u32x2*>(ep.dxv + at + cq) =
                u32x2{mm::pack_tc<TL>(g[0], g[1]), mm::pack_tc<TL>(g[2], g[3])};
        }
    }
  }
};

}  // namespace

}  // namespace skm
