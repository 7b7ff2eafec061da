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

// the lane's output e (0 .. 31) of a token, as a column after its first one
constexpr int col_of_output(int e) { return 32 * (e >> 4) + 8 * ((e & 15) >> 2) + (e & 3); }

// EpStats: part[(n0 / 256) * stride + c] = (max, sum of exp(z - max)) over the
// block's columns for listed token c; tlogit[c] = the target's logit (written
// by the one lane that holds it).
struct EpStats {
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
    const bool ragged = n - c0 < 64;  // wave-uniform
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 128 * wm + 32 * i + (lane & 31);
      const int64_t tok = m0 + row;
      const int64_t src = ep.rows[tok < m ? tok : m - 1];
      const float u = SC ? pow2f(rexp[src]) : 1.0f;
      const int tgt = target_in_wave(ep.targets[src], ep.v0 + c0, lane);
      float mx = -__builtin_inff(), sum = 0.0f;
      float z[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) z[e] = SC ? acc[i][e >> 4][e & 15] * u : acc[i][e >> 4][e & 15];
      // few waves hold a target of one of their tokens, one column block is ragged
      if (__ballot(tgt >= 0) != 0) {
        float tl = 0.0f;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (col_of_output(e) == tgt) tl = z[e];
        if (tgt >= 0 && (tgt & 4) == 0 && tok < m) ep.tlogit[tok] = tl;
      }
      if (ragged) {
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = col_of_output(e) < cols ? z[e] : -__builtin_inff();
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) mx = __builtin_fmaxf(mx, z[e]);
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float ref = mx == -__builtin_inff() ? 0.0f : mx;
#pragma unroll
      for (int e = 0; e < 32; ++e) sum += __expf(z[e] - ref);
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

// (a0, a1): four 16-bit values of columns 8 q + 4 (lane / 32) .., (b0, b1): of
// q + 1. Lanes 0 .. 31 get all eight of q, lanes 32 .. 63 of q + 1.
__device__ __forceinline__ u32x4 pair_up(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
  const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
  const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
  return u32x4{s0[0], s1[0], s0[1], s1[1]};
}

// EpGrad: dZ of the block, [listed token][ld] in up to three forms (NULL = not
// wanted): hi + lo in f16 for dLUT, scaled by head->scale 2^e of the token, and
// dxv in the tables' dtype for dX, f16 scaled by the token's own 2^e
// (xent_token_exp). f16 X: hi serves both, scaled for dLUT if there is a lo and
// else for dX. Columns n .. ld - 1 and listed rows past the count up to the next
// multiple of 32 are written as zeros. rest[c]: what rounding took from the
// target's term in dX's operand.
template <typename TX, typename TL> struct EpGrad {
  static constexpr bool OWN = __is_same(TX, bf16_t);  // dX's operand is dxv, not hi
  static constexpr bool SWAP = true, ROWS = true;
  struct Args : XentRows {
    const float* lse;    // [m]
    const float* dloss;  // [m]
    const XentHead* head;
    const int32_t* zexp;
    int64_t V, ld;
    half_t* hi;
    half_t* lo;
    TL* dxv;
    float* rest;
  };
  template <bool SC>
  static __device__ __forceinline__ void run(const f32x16 (&acc)[4][2], const Args& ep,
                                             const int32_t* __restrict__ rexp, int64_t m, int64_t n, int64_t m0,
                                             int64_t n0, int wm, int wn, int lane, int t) {
    const int64_t c0 = n0 + 64 * wn;
    const int64_t mpad = (m + 31) / 32 * 32;
    const int cols = (int)(n - c0 < 64 ? n - c0 : 64) - 4 * (lane >> 5);
    const int stored = (int)(ep.ld - c0 < 64 ? ep.ld - c0 : 64);
    const bool ragged = n - c0 < 64 || m0 + G_BM > m;  // wave-uniform
    const float scale = ep.head->scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t tok = m0 + 128 * wm + 32 * i + (lane & 31);
      if (m0 + 128 * wm + 32 * i >= mpad) break;  // wave-uniform: whole groups of 32 tokens
      const bool live = tok < m;
      const int64_t src = ep.rows[live ? tok : m - 1];
      const float u = SC ? pow2f(rexp[src]) : 1.0f;
      const int64_t target = ep.targets[src];
      const int tgt = target_in_wave(target, ep.v0 + c0, lane);
      const float lse = ep.lse[src];
      // a target outside the vocabulary gives NaN gradients (its loss is NaN)
      const float dl = target >= 0 && target < ep.V ? ep.dloss[src] : __builtin_nanf("");
      const float own = __is_same(TL, bf16_t) ? dl : dl * pow2f(xent_token_exp(dl));
      const float up = !ep.lo ? own : (ep.zexp ? dl * pow2f(ep.zexp[src]) * scale : dl * scale);
      const float dx = OWN ? own : up;
      // g[e] = dZ of output e over its row's factor. (The target's 1 and the
      // masks only where the wave has one: few waves hold a target of one of
      // their tokens, one column and one token block are ragged.)
      float g[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float z = SC ? acc[i][e >> 4][e & 15] * u : acc[i][e >> 4][e & 15];
        g[e] = __expf(z - lse);
      }
      if (__ballot(tgt >= 0) != 0) {
        float gt = 0.0f;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (col_of_output(e) == tgt) {
            g[e] -= 1.0f;
            gt = g[e];
          }
        if (ep.rest && tgt >= 0 && (tgt & 4) == 0 && live) {
          const float f = gt * dx;
          ep.rest[tok] = f - to_f32(from_f32<TL>(f));
        }
      }
      if (ragged) {
#pragma unroll
        for (int e = 0; e < 32; ++e) g[e] = col_of_output(e) < cols ? g[e] : 0.0f;
      }
      // A lane and its partner 32 lanes away hold columns 8 q .. + 3 and + 4 .. 7
      // of their token: after an exchange the lower one has all eight of an even
      // q and the upper one those of the next q, 16 bytes for one store each.
      // (ld is a multiple of 8: eight columns are stored or not together.)
      const int64_t at = tok * ep.ld + c0 + 8 * (lane >> 5);
#pragma unroll
      for (int q = 0; q < 8; q += 2) {
        const bool on = 32 * (q >> 2) + 8 * (q & 3) + 8 * (lane >> 5) < stored;
        const int64_t o = at + 32 * (q >> 2) + 8 * (q & 3);
        const float* v = g + 4 * q;  // 8 values: columns of q, then of q + 1
        if (ep.hi) {
          uint32_t h[4];
          float s[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) s[k] = live ? v[k] * up : 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = mm::pack_tc<half_t>(s[2 * k], s[2 * k + 1]);
          if (ep.lo) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              s[k] -= to_f32(__builtin_bit_cast(half_t, (uint16_t)(h[k >> 1] >> (16 * (k & 1)))));
            const u32x4 w = pair_up(mm::pack_tc<half_t>(s[0], s[1]), mm::pack_tc<half_t>(s[2], s[3]),
                                    mm::pack_tc<half_t>(s[4], s[5]), mm::pack_tc<half_t>(s[6], s[7]));
            if (on) *reinterpret_cast<u32x4*>(ep.lo + o) = w;
          }
          const u32x4 w = pair_up(h[0], h[1], h[2], h[3]);
          if (on) *reinterpret_cast<u32x4*>(ep.hi + o) = w;
        }
        if constexpr (OWN) {
          if (ep.dxv) {
            float s[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = live ? v[k] * dx : 0.0f;
            const u32x4 w = pair_up(mm::pack_tc<TL>(s[0], s[1]), mm::pack_tc<TL>(s[2], s[3]),
                                    mm::pack_tc<TL>(s[4], s[5]), mm::pack_tc<TL>(s[6], s[7]));
            if (on) *reinterpret_cast<u32x4*>(ep.dxv + o) = w;
          }
        }
      }
    }
  }
};

}  // namespace

}  // namespace skm
