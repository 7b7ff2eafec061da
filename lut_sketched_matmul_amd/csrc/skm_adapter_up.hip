// The adapters' second product, y = base + scale_s B_s h and
// dx = base_dx + D'(A_s^T dh) (skm_adapter.h).
//
// A wave takes 16 tokens (the rows of the matrix instruction) and 128
// columns at a time: column 8 c + e of the chunk is column c of instruction e, so a
// lane ends with eight consecutive columns of four tokens, 16 lanes with 256
// consecutive bytes of a row, and base and result move 16 bytes a lane. A's eight
// rows of a group are read as they lie and turned in registers. B's columns (their
// ranks are consecutive) go through LDS: read straight into operands, neighbouring
// lanes are eight columns apart and every lane is an access of its own to the L1,
// which bound the kernel (2048 tokens, 28672 columns, rank 64, 8 adapters: 121 us). Read
// in order and turned around in LDS, once for the block's four tiles of tokens, 84 us.
//
// Bound by memory and the latency that two waves per SIMD leave: 8192 x 4096, rank 16, 31 us for the 134 MB of
// base and result (4.4 TB/s; a copy of them takes 26); dx with dropout 42 us for 201 MB (4.8 TB/s). With the base of
// two chunks and the weights behind them on their way (256 registers) 36 and 47 us; three waves per SIMD (168
// registers) 33 and 51. A tile on the border between two requests takes a pass for each.
#include <type_traits>

#include "skm_adapter.h"
#include "skm_quant.h"

namespace skm {
namespace adapt {

namespace {

// The contraction of a rank in KS steps of 32. Ranks up to 16 (PACKED): one step whose
// first half takes the high terms and whose second half the low ones, so that
// one instruction does both; the weights of the halves are the same. Higher
// ranks: an instruction for each term, by the same weights.
constexpr int kPackedRank = 16;

// A's fragments of eight ranks from k0 on for the chunk's eight instructions; zeros past the rank
template <typename T>
__device__ __forceinline__ void frags_of_a(const Up& a, const T* w, int64_t col, int k0, u32x4 (&out)[8]) {
  u32x4 row[8];
  const int64_t c = col + 8 <= a.N ? col : a.N - 8;  // (those columns are not kept)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = k0 + i < a.r ? k0 + i : a.r - 1;
    row[i] = *reinterpret_cast<const u32x4*>(w + (int64_t)k * a.N + c);
  }
  if (k0 + 8 > a.r) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + i >= a.r) row[i] = kZero4;
  }
  turn8x8(row, out);
}

// B's chunk of 128 columns as pieces of eight ranks, piece p = (column p / RG, ranks 8 (p % RG) ..), taken by LW
// lanes in turn. In LDS a piece lies at slot_of: the sixteen columns c of instruction e side by side, so that a
// fragment is 16 lanes' consecutive 16 bytes, with the columns of every eighth slot permuted by XOR so that
// pieces written side by side go to different banks too.
template <int RG> __device__ __forceinline__ int slot_of(int e, int g, int c) {
  const int i = e * RG + g;
  return i * 16 + (c ^ (i & 7));
}
template <typename T, int RG, int LW, bool ALIGNED>
struct Stage {
  static constexpr int N = 128 * RG / LW;  // pieces of a lane
  u32x4 v[N];
  __device__ __forceinline__ void load(const Up& a, const T* w, int64_t ch, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = lane + LW * i, g = p % RG;
      const int64_t left = a.N - ch * 128;  // columns of the chunk
      const int c = p / RG < left ? p / RG : (int)left - 1;
      const int k0 = 8 * g < a.r ? 8 * g : 0;
      const T* q = w + (ch * 128 + c) * a.r + k0;
      if constexpr (ALIGNED) {
        v[i] = *reinterpret_cast<const u32x4*>(q);
      } else if ((ch * 128 + c) * a.r + k0 + 8 <= a.N * a.r) {
        v[i] = load_any(q);
      } else {
        v[i] = load_some(q, a.r - k0);
      }
    }
  }
  __device__ __forceinline__ void store(const Up& a, u32x4* to, int lane) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = lane + LW * i, g = p % RG, col = p / RG;
      u32x4 x = v[i];
      if constexpr (ALIGNED) {
        if (8 * g >= a.r) x = kZero4;
      } else {
        // a piece that ends behind the rank holds the next column's values there
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (8 * g + 2 * j + 1 >= a.r) x[j] &= 0xFFFFu;
          if (8 * g + 2 * j >= a.r) x[j] = 0u;
        }
      }
      to[slot_of<RG>(col & 7, g, col >> 3)] = x;
    }
  }
};

// eight columns of a row of the base as loaded: 16 bytes of T, or (backward) 32 of fp32
template <bool BACK> struct RawBase {
  u32x4 v[BACK ? 2 : 1];
};

template <typename T, bool BACK, bool ALIGNED>
__device__ __forceinline__ void load_base(const Up& a, int64_t at, RawBase<BACK>& b) {
  if constexpr (BACK) {
    b.v[0] = reinterpret_cast<const u32x4*>((const float*)a.base + at)[0];
    b.v[1] = reinterpret_cast<const u32x4*>((const float*)a.base + at)[1];
  } else if constexpr (ALIGNED) {
    b.v[0] = *reinterpret_cast<const u32x4*>((const T*)a.base + at);
  } else {
    b.v[0] = load_any((const T*)a.base + at);
  }
}

// base + v, rounded, of eight whole columns of one row
template <typename T, bool BACK, bool ALIGNED>
__device__ __forceinline__ void put8(const Up& a, int64_t at, const RawBase<BACK>& b, const float (&v)[8]) {
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (BACK) x[j] = __builtin_bit_cast(f32x4, b.v[j >> 2])[j & 3];
    else x[j] = unpack<T>(b.v[0][j >> 1], j & 1);
  }
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = pack2<T>(x[2 * j] + v[2 * j], x[2 * j + 1] + v[2 * j + 1]);
  if constexpr (BACK || ALIGNED) *reinterpret_cast<u32x4*>((T*)a.out + at) = r;
  else store_any((T*)a.out + at, r);
}

// the columns of the last vector of a row, when it is not whole
template <typename T, bool BACK>
__device__ __forceinline__ void put_some(const Up& a, int64_t at, int64_t count, const float (&v)[8]) {
  T* o = (T*)a.out + at;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < count) {
      float b = 0.f;
      if (a.base) b = BACK ? ((const float*)a.base)[at + j] : to_f32(((const T*)a.base)[at + j]);
      o[j] = from_f32<T>(b + v[j]);
    }
}

// whether the groups come out even on eight XCDs
__host__ __device__ __forceinline__ bool by_xcd(int64_t groups) { return groups % 8 == 0 || groups >= 32; }

// WT: waves of a block along the tokens, 16 each, sharing the weights; the others along the columns.
// WAL: rows of W aligned (forward: r % 8 == 0); ALIGNED: rows of base and out
// Two waves per SIMD where the operands fit their registers, else one.
template <typename T, int KS, bool PACKED, int WT, bool BACK, bool DROP, bool WAL, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES, WT > 1 ? (KS < 4 ? 2 : 1) : (KS < 2 ? 2 : 1))
void k_adapt_up(Up a, int Z, int tiles, int groups, int each) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int NT = PACKED ? 1 : 2;          // instructions of a step
  constexpr int RG = PACKED ? 2 : 4 * KS;     // groups of eight ranks
  constexpr int WC = WAVES / WT, BUFS = WT > 1 ? 2 : 1;
  const int lane = lane_id(), wave = threadIdx.x >> 6, row = lane & 15, q = lane >> 4;
  // Column groups go over the XCDs (blocks i, i + 8, .. run on one) where that leaves none of them idle: all tiles of a
  // group one after the other, so an XCD's L2 holds its columns of the weights. Else neighbouring blocks take a tile's
  // groups.
  const int at_x = (int)(blockIdx.x / 8);
  const int tile_at = by_xcd(groups) ? at_x % tiles : (int)(blockIdx.x / groups);
  const int group = by_xcd(groups) ? (int)(blockIdx.x % 8) + at_x / tiles * 8 : (int)(blockIdx.x % groups);
  if (group >= groups) return;
  const int64_t t0 = (int64_t)tile_at * (16 * WT);
  const int own = 16 * (wave % WT);  // this wave's tokens: t0 + own .. + 15
  const int zi = blockIdx.y;
  TileIds tile(a.ids, a.S, t0 + lane, lane < 16 * WT && t0 + lane < a.m);
  const uint64_t any = tile.left;
  const uint64_t here = __ballot(lane < 16 * WT && t0 + lane < a.m);

  // a wave's chunks lie side by side: where rows start anywhere, neighbouring chunks share lines (4001 x 4095, f16,
  // 34 -> 32 us)
  const int64_t all = (a.N + 127) / 128, first = ((int64_t)group * WC + wave / WT) * each;
  const int64_t chunks = first + each < all ? first + each : all;
  u32x4* lds = reinterpret_cast<u32x4*>(smem) + (wave / WT) * (BUFS * 128 * RG);
  const int stage_lane = lane + 64 * (wave % WT);
  const bool based = a.base && a.N >= 8;
  // one adapter at a time: its weights, this wave's tokens that have it, and their rows
  int adapter = 0, turn = 0, buf = 0;
  uint64_t lanes = 0;
  const T* w = nullptr;
  bool works = false, mine[4];
  int64_t at[4];
  RawBase<BACK> ahead[4];
  Stage<T, RG, 64 * WT, WAL> weights;
  auto fetch = [&](int64_t ch) {
    const int64_t col = ch * 128 + 8 * row, safe = col + 8 <= a.N ? col : 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) load_base<T, BACK, ALIGNED>(a, at[c] + safe, ahead[c]);
  };
  // the next adapter of this block, with the loads of its first chunk on their way
  auto next = [&]() {
    do {
      if (!tile.next(adapter, lanes)) return false;
    } while (turn++ % Z != zi);
    w = (const T*)a.W + (int64_t)adapter * a.r * a.N;
    const uint64_t own_lanes = (lanes >> own) & 0xFFFFu;
    // rows of other adapters read the first of this one's (and are not written)
    const int only = own_lanes ? (int)__builtin_ctzll(own_lanes) : 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int tk = 4 * q + c;
      mine[c] = (own_lanes >> tk) & 1;
      at[c] = (t0 + own + (mine[c] ? tk : only)) * a.N;
#pragma unroll
      for (int x = 0; x < (BACK ? 2 : 1); ++x) ahead[c].v[x] = kZero4;
    }
    works = own_lanes && first < chunks;
    if (!BACK && first < chunks) weights.load(a, w, first, stage_lane);
    if (works && based) fetch(first);
    return true;
  };
  bool found = next();
  if (WT == 1 && !found && zi != 0) return;  // (fewer adapters than blocks for them)

  if (a.H && group == 0 && zi == 0 && wave < WT) {
    for (int e = lane; e < 16 * a.r; e += 64) {
      const int k = e % a.r, tk = own + e / a.r;
      if (!((here >> tk) & 1)) continue;
      float v = 0.f;
      if ((any >> tk) & 1)
        for (int i = 0; i < a.splits; ++i) v += a.parts[((int64_t)i * a.m + t0 + tk) * a.rp + k];
      a.H[(t0 + tk) * a.r + k] = v;
    }
  }

  // the tokens' operands: terms of h_t times its factor
  u32x4 h[KS][NT];
  float up[4];
  {
    const int tk = own + row;
    const int id = __shfl(tile.id, tk);
    const float f = id < 0 ? 0.f : (a.scale ? a.scale[id] * a.factor : a.factor);
    float v[KS][8];
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int k0 = 8 * (PACKED ? q & 1 : 4 * s + q);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[s][j] = 0.f;
      if (id >= 0 && k0 < a.rp) {
        const float* p = a.parts + (t0 + tk) * a.rp + k0;
        // (four parts' loads on their way at once)
        for (int x0 = 0; x0 < a.splits; x0 += 4) {
          float u[4][8];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            load8<float>(p + (int64_t)(x0 + x < a.splits ? x0 + x : x0) * a.m * a.rp, u[x]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[s][j] += x0 + x < a.splits ? u[x][j] : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[s][j] *= f;
        top = fmaxf(top, fabsf(v[s][j]));
      }
    }
    int ex = 0;
    if constexpr (__is_same(T, half_t)) {
      // a power of two that brings the token's largest value into [2^14, 2^15)
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127 - 14;
      ex = e < -126 ? -126 : (e > 113 ? 113 : e);
      const float down = pow2f(-ex);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[s][j] *= down;
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4 hi, lo;
      split8<T>(v[s], hi, lo);
      if constexpr (PACKED) {
        h[s][0] = q < 2 ? hi : lo;
      } else {
        h[s][0] = hi;
        h[s][NT - 1] = lo;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) up[c] = __is_same(T, half_t) ? pow2f(__shfl(ex, 4 * q + c)) : 1.f;
  }

  const Philox g = DROP ? philox_of(a.drop.seed) : Philox{0u, 0u, 0u, 0u};
  // The next chunk's weights are fetched while one is worked on, unless a wave alone would have to hold too many.
  // (A wave's own LDS operations complete in order: it needs no barrier.)
  constexpr bool AHEAD = !BACK && (WT > 1 || KS == 1);
  while (found) {
    if constexpr (!BACK) {
      if (first < chunks) weights.store(a, lds + buf * (128 * RG), stage_lane);
      if (WT > 1) __syncthreads();
      else wave_sync();
    }
    // (all waves of a block have the same chunks when they share the weights)
    for (int64_t ch = first; ch < chunks; ++ch) {
      const bool more = ch + 1 < chunks;
      const int64_t col = ch * 128 + 8 * row;
      const bool whole = col + 8 <= a.N;
      RawBase<BACK> b[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) b[c] = ahead[c];
      if (AHEAD && more) weights.load(a, w, ch + 1, stage_lane);
      if (works) {
        f32x4 acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          u32x4 f[8];
          const int grp = PACKED ? q & 1 : 4 * s + q;
          if constexpr (BACK) {
            frags_of_a<T>(a, w, col, 8 * grp, f);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = lds[buf * (128 * RG) + slot_of<RG>(e, grp, row)];
          }
          if ((BACK || AHEAD) && s == KS - 1 && based && more) fetch(ch + 1);
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int x = NT - 1; x >= 0; --x) acc[e] = mma<T>(h[s][x], f[e], acc[e]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = acc[e][c] * up[c];
          if constexpr (DROP) {
            const u32x4 rnd = philox_block(g, (uint64_t)(at[c] + col) / 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = philox_stays(rnd, e, a.drop.threshold) ? v[e] : 0.f;
          }
          if (mine[c]) {
            if (whole) put8<T, BACK, ALIGNED>(a, at[c] + col, b[c], v);
            else if (!BACK && col < a.N) put_some<T, BACK>(a, at[c] + col, a.N - col, v);
          }
        }
      }
      if constexpr (WT > 1 && !BACK) {
        buf ^= 1;
        if (more) weights.store(a, lds + buf * (128 * RG), stage_lane);
        __syncthreads();
      } else if constexpr (!BACK) {
        wave_sync();
        if (more) {
          if (!AHEAD) weights.load(a, w, ch + 1, stage_lane);
          if (!AHEAD && works && based) fetch(ch + 1);
          weights.store(a, lds, stage_lane);
        }
        wave_sync();
      }
    }
    found = next();
  }
  // tokens without an adapter: the base alone
  const uint64_t rest = ((here & ~any) >> own) & 0xFFFFu;
  if (!rest || zi != 0 || (!BACK && a.base == a.out)) return;
  for (int64_t ch = first; ch < chunks; ++ch) {
    const int64_t col = ch * 128 + 8 * row;
    const float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int tk = 4 * q + c;
      if (!((rest >> tk) & 1)) continue;
      const int64_t at = (t0 + own + tk) * a.N + col;
      if (col + 8 <= a.N) {
        RawBase<BACK> b;
#pragma unroll
        for (int x = 0; x < (BACK ? 2 : 1); ++x) b.v[x] = kZero4;
        if (a.base) load_base<T, BACK, ALIGNED>(a, at, b);
        put8<T, BACK, ALIGNED>(a, at, b, v);
      } else if (col < a.N) {
        put_some<T, BACK>(a, at, a.N - col, v);
      }
    }
  }
}

}  // namespace

hipError_t launch_up(const Up& a, int dtype, bool back, hipStream_t s) {
  const int64_t chunks = (a.N + 127) / 128;
  auto go = [&](auto t, auto ks, auto packed, auto wt, auto bk, auto drop, auto wal, auto al) {
    typedef typename decltype(t)::type T;
    constexpr int WT = decltype(wt)::value, WC = WAVES / WT, KS = decltype(ks)::value;
    constexpr bool BACK = decltype(bk)::value, PACKED = decltype(packed)::value;
    constexpr size_t lds = BACK ? 0 : size_t(WT > 1 ? 2 : WC) * 128 * (PACKED ? 2 : 4 * KS) * 16;
    const auto kern = k_adapt_up<T, KS, PACKED, WT, BACK, decltype(drop)::value, decltype(wal)::value, decltype(al)::value>;
    static const hipError_t ready = prepare_kernel((const void*)kern, lds);
    if (ready != hipSuccess) return ready;
    const int64_t tiles = (a.m + 16 * WT - 1) / (16 * WT);
    // Blocks: as many as run at once (two per CU), or twice that where they are many, then several chunks to a wave, whose
    // operands serve all of them. A few tiles (decoding) may hold an adapter per token: a block for each. Up to 256
    // tokens may be some of both: four blocks (128 tokens with 64 adapters, 4096 -> 11008 at rank 16, 33 -> 26 us; 128
    // of 8 requests 9.1 either way). More are requests of many tokens, and a block walks its tile's adapters.
    const int most = a.S < 16 * WT ? a.S : 16 * WT;
    const int64_t Z = WT > 1 || tiles > 16 ? 1 : (tiles <= 4 || most < 4 ? most : 4);
    int64_t want = WT == 1 && tiles <= 4 ? 512 / (tiles * Z) : 1024 / tiles;
    if (want < 1) want = 1;
    if (want > 8) want = want / 8 * 8;
    const int64_t each = (chunks + WC * want - 1) / (WC * want);  // chunks of a wave
    const int64_t groups = (chunks + WC * each - 1) / (WC * each);
    const int64_t blocks = (by_xcd(groups) ? (groups + 7) / 8 * 8 : groups) * tiles;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks, (unsigned)Z), dim3(64 * WAVES), lds, s, a, (int)Z, (int)tiles,
                       (int)groups, (int)each);
    return hipGetLastError();
  };
  std::true_type yes;
  std::false_type no;
  auto with_form = [&](auto t, auto ks, auto pk, auto wt) {
    if (back) return a.drop.threshold ? go(t, ks, pk, wt, yes, yes, yes, yes) : go(t, ks, pk, wt, yes, no, yes, yes);
    if (a.N % 8 == 0) return a.r % 8 == 0 ? go(t, ks, pk, wt, no, no, yes, yes) : go(t, ks, pk, wt, no, no, no, yes);
    return a.r % 8 == 0 ? go(t, ks, pk, wt, no, no, yes, no) : go(t, ks, pk, wt, no, no, no, no);
  };
  auto with_tiles = [&](auto t, auto ks, auto pk) {
    if (a.m > kManyTokens) return with_form(t, ks, pk, std::integral_constant<int, WAVES>{});
    return with_form(t, ks, pk, std::integral_constant<int, 1>{});
  };
  auto with_steps = [&](auto t) {
    std::integral_constant<int, 1> one;
    if (a.r <= kPackedRank) return with_tiles(t, one, yes);
    if (a.r <= 32) return with_tiles(t, one, no);
    if (a.r <= 64) return with_tiles(t, std::integral_constant<int, 2>{}, no);
    return with_tiles(t, std::integral_constant<int, 4>{}, no);
  };
  if (dtype == DT_F16) return with_steps(dtype_of<DT_F16>{});
  return with_steps(dtype_of<DT_BF16>{});
}

}  // namespace adapt
}  // namespace skm
