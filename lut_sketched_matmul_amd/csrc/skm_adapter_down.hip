// The adapters' first product, h = A_s D(x) and dh = B_s^T dy (skm_adapter.h).
//
// A block takes 16 TT tokens, one range of the contraction and (of the distinct
// adapters in the tile) every Z-th; its waves take turns over 64 columns of that
// range and add up in LDS. Fragments come straight from memory, 16 bytes a
// lane; with dropout each of X's fragments is one generator call.
//
// Few tokens are split along the contraction until the launch has about 512
// blocks, and over the adapters: one token of 4096 columns is 16 blocks of 256
// columns. The splits' sums are added by their reader, in order.
#include <type_traits>

#include "skm_adapter.h"

namespace skm {
namespace adapt {

namespace {

// P's and W's fragments of 64 columns from k on, and their products
template <typename T, int TT, int RT, bool DROP, bool WHOLE, bool ALIGNED>
__device__ __forceinline__ void down_chunk(const T* const (&p)[TT], const T* const (&w)[RT], const uint64_t (&block)[TT],
                                           int64_t k, int64_t K, const Philox& g, uint32_t threshold,
                                           f32x4 (&acc)[TT][RT]) {
  u32x4 x[2][TT], y[2][RT];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t at = k + 32 * u;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      if constexpr (WHOLE) x[u][i] = ALIGNED ? *reinterpret_cast<const u32x4*>(p[i] + at) : load_any(p[i] + at);
      else x[u][i] = load_some(p[i] + at, K - at);
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      if constexpr (WHOLE) y[u][j] = *reinterpret_cast<const u32x4*>(w[j] + at);
      else y[u][j] = load_some(w[j] + at, K - at);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if constexpr (DROP) {
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const u32x4 rnd = philox_block(g, block[i] + (uint64_t)(k + 32 * u) / 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[u][i][j] = philox_mask2(rnd, j, threshold, x[u][i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = mma<T>(x[u][i], y[u][j], acc[i][j]);
  }
}

template <typename T, int TT, int RT, bool DROP, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES) void k_adapt_down(Down a, int Z, float factor) {
  extern __shared__ __align__(16) unsigned char smem[];
  f32x4* sums = reinterpret_cast<f32x4*>(smem);  // [WAVES][TT][RT][64]
  const int lane = lane_id(), wave = threadIdx.x >> 6, row = lane & 15, q = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TT);
  const int zi = blockIdx.z % Z, r0 = (blockIdx.z / Z) * (16 * RT);
  const int64_t kb = (int64_t)blockIdx.y * a.per;
  const int64_t ke = kb + a.per < a.K ? kb + a.per : a.K;
  const Philox g = DROP ? philox_of(a.drop.seed) : Philox{0u, 0u, 0u, 0u};

  const T* p[TT];
  uint64_t block[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    int64_t t = t0 + 16 * i + row;
    if (t >= a.m) t = a.m - 1;  // (its row is not kept)
    p[i] = (const T*)a.P + t * a.K + 8 * q;
    block[i] = (uint64_t)(t * a.K) / 8 + q;
  }
  TileIds tile(a.ids, a.S, t0 + lane, lane < 16 * TT && t0 + lane < a.m);
  int adapter, turn = 0;
  uint64_t lanes;
  while (tile.next(adapter, lanes)) {
    if (turn++ % Z != zi) continue;
    const T* w[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      int k = r0 + 16 * j + row;
      if (k >= a.r) k = a.r - 1;  // (its column is not kept)
      w[j] = (const T*)a.W + adapter * a.wstride + k * a.ldw + 8 * q;
    }
    f32x4 acc[TT][RT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t stride = 64 * WAVES;
    int64_t k = kb + 64 * wave;
    for (; k + 64 <= ke; k += stride)
      down_chunk<T, TT, RT, DROP, true, ALIGNED>(p, w, block, k, a.K - 8 * q, g, a.drop.threshold, acc);
    if (k < ke) down_chunk<T, TT, RT, DROP, false, ALIGNED>(p, w, block, k, a.K - 8 * q, g, a.drop.threshold, acc);

    __syncthreads();  // (the last adapter's sums are still read)
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) sums[((wave * TT + i) * RT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int e = threadIdx.x; e < TT * RT * 64; e += 64 * WAVES) {
      f32x4 v = sums[e];
#pragma unroll
      for (int x = 1; x < WAVES; ++x) v += sums[x * TT * RT * 64 + e];
      const int l = e & 63, j = (e >> 6) % RT, i = (e >> 6) / RT;
      const int k = r0 + 16 * j + (l & 15);
      if (k < a.rp) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int tk = 16 * i + 4 * (l >> 4) + c;
          if ((lanes >> tk) & 1)
            a.parts[((int64_t)blockIdx.y * a.m + t0 + tk) * a.rp + k] = k < a.r ? v[c] * factor : 0.f;
        }
      }
    }
  }
}

}  // namespace

// Ranges of the contraction: as many as bring the launch to 512 blocks, of at least 256 columns (one chunk
// per wave).
int down_splits(int64_t m, int64_t K, int S, int64_t& per) {
  const int64_t tiles = (m + 15) / 16, adapters = S < m ? (S < 16 ? S : 16) : (m < 16 ? m : 16);
  int64_t want = 512 / (tiles * adapters);
  const int64_t most = (K + 255) / 256;
  if (want > most) want = most;
  if (want < 1) want = 1;
  per = ((K + want - 1) / want + 63) / 64 * 64;
  return (int)((K + per - 1) / per);
}

hipError_t launch_down(const Down& a, int dtype, hipStream_t s) {
  // the share that stays divides the sums: one multiplication per sum instead of one per value
  const float factor = a.drop.threshold ? a.drop.inv() : 1.f;
  auto go = [&](auto t, auto tt, auto rt, auto drop, auto aligned) {
    typedef typename decltype(t)::type T;
    constexpr int TT = decltype(tt)::value, RT = decltype(rt)::value;
    const int64_t tiles = (a.m + 16 * TT - 1) / (16 * TT);
    const int most = a.S < 16 * TT ? a.S : 16 * TT;
    int64_t Z = 1024 / (tiles * a.splits);
    if (Z > most) Z = most;
    if (Z < 1) Z = 1;
    const int groups = (a.r + 16 * RT - 1) / (16 * RT);
    hipLaunchKernelGGL((k_adapt_down<T, TT, RT, decltype(drop)::value, decltype(aligned)::value>),
                       dim3((unsigned)tiles, (unsigned)a.splits, (unsigned)(Z * groups)), dim3(64 * WAVES),
                       WAVES * TT * RT * 64 * 16, s, a, (int)Z, factor);
    return hipGetLastError();
  };
  auto with_ranks = [&](auto t, auto tt, auto drop, auto aligned) {
    if (a.r <= 16) return go(t, tt, std::integral_constant<int, 1>{}, drop, aligned);
    if (a.r <= 32) return go(t, tt, std::integral_constant<int, 2>{}, drop, aligned);
    return go(t, tt, std::integral_constant<int, 4>{}, drop, aligned);
  };
  auto with_rest = [&](auto t) {
    // two row tiles share a wave's weights from 4096 tokens on: 256 blocks of 16 tokens fill the CUs alone
    std::integral_constant<int, 1> one;
    std::integral_constant<int, 2> two;
    std::true_type yes;
    std::false_type no;
    if (a.drop.threshold) return a.m >= 4096 ? with_ranks(t, two, yes, yes) : with_ranks(t, one, yes, yes);
    if (a.K % 8 == 0) return a.m >= 4096 ? with_ranks(t, two, no, yes) : with_ranks(t, one, no, yes);
    return a.m >= 4096 ? with_ranks(t, two, no, no) : with_ranks(t, one, no, no);
  };
  if (dtype == DT_F16) return with_rest(dtype_of<DT_F16>{});
  return with_rest(dtype_of<DT_BF16>{});
}

}  // namespace adapt
}  // namespace skm
