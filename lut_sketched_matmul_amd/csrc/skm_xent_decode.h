// Cross entropy of few tokens: the decode kernel (skm_decode.h) ends in softmax
// statistics (EpDecodeStats) or in the logits' gradient (EpDecodeGrad). It
// reads the indices once per 16 tokens, where the 256-token tiles would spend
// most of their matrix work on padding.
#pragma once

#include "skm_decode.h"
#include "skm_xent.h"

namespace skm {

namespace {

// part[t0 + token][block] = (max, sum of exp(z - max)) over the block's 16 words
struct EpDecodeStats {
  static constexpr bool GROUPS = true;
  struct Args {
    const int64_t* targets;  // [m]
    float2* part;
    int64_t blocks;
    float* tlogit;
    int64_t t0;
  };
  static __device__ __forceinline__ void put(const Args& ep, bool ok, int token, int64_t row, float v, int m,
                                             int64_t n) {
    const float z = ok ? v : -__builtin_inff();
    float mx = z;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, o, 64));
    const float ref = mx == -__builtin_inff() ? 0.0f : mx;
    float sum = ok ? __expf(z - ref) : 0.0f;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (token >= m) return;
    if (row % DEC_ROWS == 0) ep.part[(ep.t0 + token) * ep.blocks + row / DEC_ROWS] = float2{mx, sum};
    if (ok && ep.targets[ep.t0 + token] == row) ep.tlogit[ep.t0 + token] = v;
  }
};

// dZ of the listed tokens among t0 .. t0 + m - 1, in the forms of EpGrad;
// the first group also writes the zero rows that pad the list
template <typename TX, typename TL> struct EpDecodeGrad {
  static constexpr bool GROUPS = true;
  static constexpr bool OWN = __is_same(TX, bf16_t);
  struct Args {
    const int32_t* pos;  // listed row of every token, -1 = ignored
    const XentHead* head;
    const int64_t* targets;
    const float* lse;
    const float* dloss;
    const int32_t* zexp;
    int64_t V, v0, ld, t0;
    half_t* hi;
    half_t* lo;
    TL* dxv;
    float* rest;
  };
  // dZ as dLUT's forms and dX's hold it
  static __device__ __forceinline__ void store(const Args& ep, int64_t at, float up, float dx) {
    if (ep.hi) {
      const half_t h = from_f32<half_t>(up);
      ep.hi[at] = h;
      if (ep.lo) ep.lo[at] = from_f32<half_t>(up - to_f32(h));
    }
    if (OWN && ep.dxv) ep.dxv[at] = from_f32<TL>(dx);
  }
  static __device__ __forceinline__ void put(const Args& ep, bool ok, int token, int64_t row, float v, int m,
                                             int64_t n) {
    if (row >= ep.ld) return;
    if (ep.t0 == 0) {
      const int64_t count = ep.head->count, pad = (count + 31) / 32 * 32;
      for (int64_t c = count + token; c < pad; c += 16) store(ep, c * ep.ld + row, 0.0f, 0.0f);
    }
    if (token >= m) return;
    const int64_t t = ep.t0 + token;
    const int64_t c = ep.pos[t];
    if (c < 0) return;
    const int64_t target = ep.targets[t];
    const float dl = target >= 0 && target < ep.V ? ep.dloss[t] : __builtin_nanf("");
    const float own = __is_same(TL, bf16_t) ? dl : dl * pow2f(xent_token_exp(dl));
    const float up =
        !ep.lo ? own : (ep.zexp ? dl * pow2f(ep.zexp[t]) * ep.head->scale : dl * ep.head->scale);
    const float dx = OWN ? own : up;
    const bool mine = ok && ep.v0 + row == target;
    const float p = __expf(v - ep.lse[t]) - (mine ? 1.0f : 0.0f);
    store(ep, c * ep.ld + row, ok ? p * up : 0.0f, ok ? p * dx : 0.0f);
    if (mine && ep.rest) ep.rest[c] = p * dx - to_f32(from_f32<TL>(p * dx));
  }
};

// All m tokens in one launch, 16 per block. The vocabulary has many 16-row
// blocks: 8 waves each, two or more blocks per CU (as the plain decode above 384
// blocks)
template <int B, typename TX, typename TL, typename EP>
hipError_t xent_decode(const XentGemm& g, const typename EP::Args& ep, hipStream_t s) {
  const Problem& p = g.p;
  const TX* X = (const TX*)g.X;
  const TL* lut = (const TL*)g.lut;
  const uint32_t ug = (uint32_t)(p.group_cols() / 32);
  const uint32_t magic = ug == 1 ? 0u : (uint32_t)((((uint64_t)1) << 32) / ug + 1);
  SetArgs sa;
  sa.rexp = g.rexp;
  const bool xl = xent_decode_stages(p), xt = !xl && p.m >= DEC_XT_MIN_M;
  if (p.units() % 4 != 0)
    return xl ? decode_launch<B, 8, TX, TL, true, true, false, EP>(X, g.idx, lut, p, ep, s, magic, sa)
              : (xt ? decode_launch<B, 8, TX, TL, true, false, true, EP>(X, g.idx, lut, p, ep, s, magic, sa)
                    : decode_launch<B, 8, TX, TL, true, false, false, EP>(X, g.idx, lut, p, ep, s, magic, sa));
  return xl ? decode_launch<B, 8, TX, TL, false, true, false, EP>(X, g.idx, lut, p, ep, s, magic, sa)
            : (xt ? decode_launch<B, 8, TX, TL, false, false, true, EP>(X, g.idx, lut, p, ep, s, magic, sa)
                  : decode_launch<B, 8, TX, TL, false, false, false, EP>(X, g.idx, lut, p, ep, s, magic, sa));
}

}  // namespace

}  // namespace skm
