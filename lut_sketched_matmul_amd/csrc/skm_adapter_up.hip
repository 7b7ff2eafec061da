// The adapters' second product, y = base + scale_s B_s h and
// dx = base_dx + D'(A_s^T dh) (skm_adapter.h).
//
// A wave takes 16 TT tokens (the rows of the matrix instruction) and 128
// columns at a time: column 8 c + e of the chunk is column c of instruction e, so a
// lane ends with eight consecutive columns of four tokens, 16 lanes with 256
// consecutive bytes of a row, and base and result move 16 bytes a lane. B is read
// as it lies (a column's ranks are consecutive); A's eight rows of a group are
// turned in registers.
#include <type_traits>

#include "skm_adapter.h"
#include "skm_quant.h"

namespace skm {
namespace adapt {

namespace {

constexpr int TERMS = 2;

// fragments of eight ranks (group grp of `groups` along the contraction) for the chunk's eight instructions
template <typename T, bool BACK, bool ALIGNED>
__device__ __forceinline__ void weight_frags(const Up& a, const T* w, int64_t col, int grp, int groups,
                                             u32x4 (&out)[8]) {
  const bool live = grp < TERMS * groups;
  const int k0 = 8 * (grp % groups);
  if constexpr (BACK) {
    u32x4 row[8];
    const int64_t c = col + 8 <= a.N ? col : a.N - 8;  // (those columns are not kept)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + i < a.r ? k0 + i : a.r - 1;
      row[i] = *reinterpret_cast<const u32x4*>(w + (int64_t)k * a.N + c);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!live || k0 + i >= a.r) row[i] = kZero4;
    turn8x8(row, out);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = col + e < a.N ? col + e : a.N - 1;
      const T* p = w + c * a.r + k0;
      if constexpr (ALIGNED) {
        out[e] = *reinterpret_cast<const u32x4*>(p);
      } else {
        // a group that ends behind the rank reads into the next column's, the last one value by value
        if (c * a.r + k0 + 8 <= a.N * a.r) out[e] = load_any(p);
        else out[e] = load_some(p, a.r - k0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (k0 + 2 * j + 1 >= a.r) out[e][j] &= 0xFFFFu;
          if (k0 + 2 * j >= a.r) out[e][j] = 0u;
        }
      }
      if (!live) out[e] = kZero4;
    }
  }
}

// base + v, rounded, of eight columns of one row
template <typename T, bool BACK, bool ALIGNED>
__device__ __forceinline__ void put8(const Up& a, int64_t t, int64_t col, const float (&v)[8]) {
  const int64_t at = t * a.N + col;
  T* o = (T*)a.out + at;
  if (col + 8 <= a.N) {
    float b[8];
    if constexpr (BACK) {
      if (a.base) load8<float>((const float*)a.base + at, b);
    } else if (a.base) {
      const u32x4 raw = ALIGNED ? *reinterpret_cast<const u32x4*>((const T*)a.base + at)
                                : load_any((const T*)a.base + at);
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = unpack<T>(raw[j >> 1], j & 1);
    }
    if (!a.base) {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = 0.f;
    }
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = pack2<T>(b[2 * j] + v[2 * j], b[2 * j + 1] + v[2 * j + 1]);
    if constexpr (BACK || ALIGNED) *reinterpret_cast<u32x4*>(o) = r;
    else store_any(o, r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < a.N) {
        float b = 0.f;
        if (a.base) b = BACK ? ((const float*)a.base)[at + j] : to_f32(((const T*)a.base)[at + j]);
        o[j] = from_f32<T>(b + v[j]);
      }
  }
}

// KS steps of 32 along ranks x terms; WAL: rows of W aligned (forward: r % 8 == 0); ALIGNED: rows of base and out
template <typename T, int KS, int TT, bool BACK, bool DROP, bool WAL, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES) void k_adapt_up(Up a, int Z) {
  const int lane = lane_id(), wave = threadIdx.x >> 6, row = lane & 15, q = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TT);
  const int zi = blockIdx.z, groups = a.rp / 8;
  TileIds tile(a.ids, a.S, t0 + lane, lane < 16 * TT && t0 + lane < a.m);
  const uint64_t any = tile.left;
  const uint64_t here = __ballot(lane < 16 * TT && t0 + lane < a.m);

  if (a.H && blockIdx.y == 0 && blockIdx.z == 0) {
    for (int e = threadIdx.x; e < 16 * TT * a.r; e += 64 * WAVES) {
      const int tk = e / a.r, k = e - tk * a.r;
      if (!((here >> tk) & 1)) continue;
      float v = 0.f;
      if ((any >> tk) & 1)
        for (int i = 0; i < a.splits; ++i) v += a.parts[((int64_t)i * a.m + t0 + tk) * a.rp + k];
      a.H[(t0 + tk) * a.r + k] = v;
    }
  }

  // the tokens' operands: terms of h_t times its factor
  u32x4 h[TT][KS];
  int ex[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int tk = 16 * i + row;
    const int id = __shfl(tile.id, tk);
    const float f = id < 0 ? 0.f : (a.scale ? a.scale[id] * a.factor : a.factor);
    float v[KS][8];
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int grp = 4 * s + q;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[s][j] = 0.f;
      if (id >= 0 && grp < TERMS * groups) {
        const float* p = a.parts + (t0 + tk) * a.rp + 8 * (grp % groups);
        for (int x = 0; x < a.splits; ++x) {
          float u[8];
          load8<float>(p + (int64_t)x * a.m * a.rp, u);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[s][j] += u[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[s][j] *= f;
        top = fmaxf(top, fabsf(v[s][j]));
      }
    }
    ex[i] = 0;
    if constexpr (__is_same(T, half_t)) {
      // a power of two that brings the token's largest value into [2^14, 2^15)
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127 - 14;
      ex[i] = e < -126 ? -126 : (e > 113 ? 113 : e);
      const float down = pow2f(-ex[i]);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[s][j] *= down;
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = v[s][j];
      const u32x4 lo = term_of<T>(u, 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = v[s][j];
      h[i][s] = 4 * s + q < groups ? term_of<T>(u, 0) : lo;
    }
  }
  float up[TT][4];
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) up[i][c] = __is_same(T, half_t) ? pow2f(__shfl(ex[i], 4 * q + c)) : 1.f;

  const Philox g = DROP ? philox_of(a.drop.seed) : Philox{0u, 0u, 0u, 0u};
  const int64_t chunks = (a.N + 127) / 128;
  const int64_t first = (int64_t)blockIdx.y * WAVES + wave, step = (int64_t)gridDim.y * WAVES;
  int adapter, turn = 0;
  uint64_t lanes;
  while (tile.next(adapter, lanes)) {
    if (turn++ % Z != zi) continue;
    const T* w = (const T*)a.W + (int64_t)adapter * a.r * a.N;
    for (int64_t ch = first; ch < chunks; ch += step) {
      const int64_t col = ch * 128 + 8 * row;
      f32x4 acc[TT][8];
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        u32x4 f[8];
        weight_frags<T, BACK, WAL>(a, w, col, 4 * s + q, groups, f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int i = 0; i < TT; ++i) acc[i][e] = mma<T>(h[i][s], f[e], acc[i][e]);
      }
      if (col < a.N) {
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int tk = 16 * i + 4 * q + c;
            if (!((lanes >> tk) & 1)) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = acc[i][e][c] * up[i][c];
            if constexpr (DROP) {
              const u32x4 rnd = philox_block(g, (uint64_t)((t0 + tk) * a.N + col) / 8);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = philox_stays(rnd, e, a.drop.threshold) ? v[e] : 0.f;
            }
            put8<T, BACK, ALIGNED>(a, t0 + tk, col, v);
          }
      }
    }
  }
  // tokens without an adapter: the base alone
  const uint64_t rest = here & ~any;
  if (!rest || zi != 0 || (!BACK && a.base == a.out)) return;
  for (int64_t ch = first; ch < chunks; ch += step) {
    const int64_t col = ch * 128 + 8 * row;
    if (col >= a.N) continue;
    const float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int tk = 16 * i + 4 * q + c;
        if ((rest >> tk) & 1) put8<T, BACK, ALIGNED>(a, t0 + tk, col, v);
      }
  }
}

}  // namespace

hipError_t launch_up(const Up& a, int dtype, bool back, hipStream_t s) {
  const int64_t chunks = (a.N + 127) / 128;
  auto go = [&](auto t, auto ks, auto tt, auto bk, auto drop, auto wal, auto al) {
    typedef typename decltype(t)::type T;
    constexpr int TT = decltype(tt)::value;
    const int64_t tiles = (a.m + 16 * TT - 1) / (16 * TT);
    int64_t gy = (chunks + WAVES - 1) / WAVES;
    // enough waves for every SIMD, then several chunks to a wave: its tokens' operands serve all of them
    const int64_t want = 2048 / tiles;
    if (gy > want) gy = want < 1 ? 1 : want;
    const int most = a.S < 16 * TT ? a.S : 16 * TT;
    int64_t Z = 1024 / (tiles * gy);
    if (Z > most) Z = most;
    if (Z < 1) Z = 1;
    hipLaunchKernelGGL((k_adapt_up<T, decltype(ks)::value, TT, decltype(bk)::value, decltype(drop)::value,
                                   decltype(wal)::value, decltype(al)::value>),
                       dim3((unsigned)tiles, (unsigned)gy, (unsigned)Z), dim3(64 * WAVES), 0, s, a, (int)Z);
    return hipGetLastError();
  };
  std::true_type yes;
  std::false_type no;
  auto with_form = [&](auto t, auto ks, auto tt) {
    if (back) return a.drop.threshold ? go(t, ks, tt, yes, yes, yes, yes) : go(t, ks, tt, yes, no, yes, yes);
    if (a.N % 8 == 0) return a.r % 8 == 0 ? go(t, ks, tt, no, no, yes, yes) : go(t, ks, tt, no, no, no, yes);
    return a.r % 8 == 0 ? go(t, ks, tt, no, no, yes, no) : go(t, ks, tt, no, no, no, no);
  };
  auto with_steps = [&](auto t) {
    std::integral_constant<int, 1> one;
    const int ks = (TERMS * (a.rp / 8) + 3) / 4;
    if (a.m >= 4096) {
      std::integral_constant<int, 2> two;
      if (ks <= 1) return with_form(t, one, two);
      if (ks <= 2) return with_form(t, two, two);
      if (ks <= 4) return with_form(t, std::integral_constant<int, 4>{}, two);
      return with_form(t, std::integral_constant<int, 8>{}, two);
    }
    if (ks <= 1) return with_form(t, one, one);
    if (ks <= 2) return with_form(t, std::integral_constant<int, 2>{}, one);
    if (ks <= 4) return with_form(t, std::integral_constant<int, 4>{}, one);
    return with_form(t, std::integral_constant<int, 8>{}, one);
  };
  if (dtype == DT_F16) return with_steps(dtype_of<DT_F16>{});
  return with_steps(dtype_of<DT_BF16>{});
}

}  // namespace adapt
}  // namespace skm
