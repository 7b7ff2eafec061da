// The adapters' first product, h = A_s D(x) and dh = B_s^T dy (skm_adapter.h).
//
// Three kernels, a wave with 16 tokens in each:
//   k_adapt_down        up to kManyTokens tokens. A block takes 16 tokens, one range
//                       of the contraction and (of the distinct adapters in the tile)
//                       every Z-th; its waves take turns over 64 columns of that range
//                       and add up in LDS. Fragments come straight from memory, 16
//                       bytes a lane.
//   k_adapt_down_lds    more tokens, ranks up to kSharedRank: the same tile, 128 columns
//                       at a time through LDS of the wave's own.
//   k_adapt_down_tiles  more tokens and ranks: 64 tokens a block, whose waves share
//                       the weights in LDS.
// With dropout each of X's fragments is one generator call.
//
// Few tokens are split along the contraction until the launch has about 512
// blocks, and over the adapters: 64 tokens of 4096 columns with 64 adapters are 8
// ranges and 16 blocks for a tile's adapters, 5.8 us. (Most calls of a few tokens
// with rank <= 32 and no dropout do not come here: skm_adapter_few.hip.) The ranges'
// sums are added by their reader, in order.
//
// Many tokens: 8192 x 4096, rank 16, 18.4 us (3.7 TB/s of a read that a copy's rate would do in 12), with dropout
// 19.8; what is left is the start and the end of 512 blocks that all run at once.
#include <type_traits>

#include "skm_adapter.h"

namespace skm {
namespace adapt {

namespace {

// P's and W's fragments of 64 columns from k on, and their products
template <typename T, int RT, bool DROP, bool WHOLE, bool ALIGNED>
__device__ __forceinline__ void down_chunk(const T* p, const T* const (&w)[RT], uint64_t block, int64_t k, int64_t K,
                                           const Philox& g, const PhiloxMask& mask, f32x4 (&acc)[RT]) {
  u32x4 x[2], y[2][RT];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t at = k + 32 * u;
    if constexpr (WHOLE) x[u] = ALIGNED ? *reinterpret_cast<const u32x4*>(p + at) : load_any(p + at);
    else x[u] = load_some(p + at, K - at);
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      if constexpr (WHOLE) y[u][j] = *reinterpret_cast<const u32x4*>(w[j] + at);
      else y[u][j] = load_some(w[j] + at, K - at);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if constexpr (DROP) {
      const u32x4 rnd = philox_block(g, block + (uint64_t)(k + 32 * u) / 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[u][j] = philox_mask2(rnd[j], mask, x[u][j]);
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = mma<T>(x[u], y[u][j], acc[j]);
  }
}

template <typename T, int RT, bool DROP, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES) void k_adapt_down(Down a, int Z, float factor) {
  extern __shared__ __align__(16) unsigned char smem[];
  f32x4* sums = reinterpret_cast<f32x4*>(smem);  // [WAVES][RT][64]
  const int lane = lane_id(), wave = threadIdx.x >> 6, row = lane & 15, q = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int zi = blockIdx.z % Z, r0 = (blockIdx.z / Z) * (16 * RT);
  const int64_t kb = (int64_t)blockIdx.y * a.per;
  const int64_t ke = kb + a.per < a.K ? kb + a.per : a.K;
  const Philox g = DROP ? philox_of(a.drop.seed) : Philox{0u, 0u, 0u, 0u};
  const PhiloxMask mask = philox_mask_of(a.drop.threshold);

  const int64_t t = t0 + row < a.m ? t0 + row : a.m - 1;  // (a row past the last is not kept)
  const T* p = (const T*)a.P + t * a.K + 8 * q;
  const uint64_t block = (uint64_t)(t * a.K) / 8 + q;
  TileIds tile(a.ids, a.S, t0 + lane, lane < 16 && t0 + lane < a.m);
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
    f32x4 acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t stride = 64 * WAVES;
    int64_t k = kb + 64 * wave;
    for (; k + 64 <= ke; k += stride)
      down_chunk<T, RT, DROP, true, ALIGNED>(p, w, block, k, a.K - 8 * q, g, mask, acc);
    if (k < ke) down_chunk<T, RT, DROP, false, ALIGNED>(p, w, block, k, a.K - 8 * q, g, mask, acc);

    __syncthreads();  // (the last adapter's sums are still read)
#pragma unroll
    for (int j = 0; j < RT; ++j) sums[(wave * RT + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * 64; e += 64 * WAVES) {
      f32x4 v = sums[e];
#pragma unroll
      for (int x = 1; x < WAVES; ++x) v += sums[x * RT * 64 + e];
      const int l = e & 63, k2 = r0 + 16 * (e >> 6) + (l & 15);
      if (k2 >= a.rp) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int tk = 4 * (l >> 4) + c;
        if ((lanes >> tk) & 1)
          a.parts[((int64_t)blockIdx.y * a.m + t0 + tk) * a.rp + k2] = k2 < a.r ? v[c] * factor : 0.f;
      }
    }
  }
}

// The same through LDS, for many tokens: loaded straight into operands, neighbouring lanes are rows apart and every
// lane is an access of its own to the L1 (8192 tokens of 4095 columns, not whole vectors: 35 us). Here 16 lanes read 256
// consecutive bytes and a wave turns its 128 columns around in LDS of its own; the next 128 are on their way
// meanwhile. A row's 16 pieces are permuted by XOR with its number, so that the 16 rows of an operand lie in
// different banks. Dropout's generator works on the pieces as they were loaded.
template <typename T, int RT, bool DROP, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES) void k_adapt_down_lds(Down a, float factor) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int COLS = 128;
  const int lane = lane_id(), wave = threadIdx.x >> 6, row = lane & 15, q = lane >> 4;
  u32x4* lds = reinterpret_cast<u32x4*>(smem) + wave * (1 + RT) * 256;  // the wave's tokens, then its weights
  f32x4* sums = reinterpret_cast<f32x4*>(smem);                         // (at the end) [WAVES][RT][64]
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int r0 = blockIdx.z * (16 * RT);
  const int64_t kb = (int64_t)blockIdx.y * a.per;
  const int64_t ke = kb + a.per < a.K ? kb + a.per : a.K;
  const Philox g = DROP ? philox_of(a.drop.seed) : Philox{0u, 0u, 0u, 0u};
  const PhiloxMask mask = philox_mask_of(a.drop.threshold);

  // this lane's pieces: columns 8 row .. of rows 4 i + q
  int64_t prow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + 4 * i + q;
    prow[i] = (t < a.m ? t : a.m - 1) * a.K;  // (a row past the last is not kept)
  }
  TileIds tile(a.ids, a.S, t0 + lane, lane < 16 && t0 + lane < a.m);
  int adapter;
  uint64_t lanes;
  while (tile.next(adapter, lanes)) {
    const T* w = (const T*)a.W + adapter * a.wstride;
    u32x4 x[4], y[4 * RT];
    auto load = [&](int64_t k) {
      const int64_t at = k + 8 * row, left = a.K - at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const T* p = (const T*)a.P + prow[i] + at;
        if (ALIGNED) x[i] = left > 0 ? *reinterpret_cast<const u32x4*>(p) : kZero4;  // (K is whole pieces)
        else x[i] = left >= 8 ? load_any(p) : load_some(p, left);
      }
#pragma unroll
      for (int i = 0; i < 4 * RT; ++i) {
        int r = r0 + 4 * i + q;
        if (r >= a.r) r = a.r - 1;  // (its column is not kept)
        // (the rows of W are whole pieces, padded with zeros where P's are not)
        y[i] = left > 0 ? *reinterpret_cast<const u32x4*>(w + r * a.ldw + at) : kZero4;
      }
    };
    auto store = [&](int64_t k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + q;
        if constexpr (DROP) {
          const u32x4 rnd = philox_block(g, (uint64_t)(prow[i] + k + 8 * row) / 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i][j] = philox_mask2(rnd[j], mask, x[i][j]);
        }
        lds[r * 16 + (row ^ r)] = x[i];
      }
#pragma unroll
      for (int i = 0; i < 4 * RT; ++i) {
        const int r = 4 * i + q;
        lds[256 + r * 16 + (row ^ (r & 15))] = y[i];
      }
    };
    f32x4 acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int64_t k = kb + COLS * wave;
    if (k < ke) load(k);
    __syncthreads();  // (the last adapter's sums are still read)
    for (; k < ke; k += COLS * WAVES) {
      // (a wave's LDS operations complete in order: no barrier between its own)
      store(k);
      wave_sync();
      if (k + COLS * WAVES < ke) load(k + COLS * WAVES);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const u32x4 p = lds[row * 16 + ((4 * s + q) ^ row)];
#pragma unroll
        for (int j = 0; j < RT; ++j)
          acc[j] = mma<T>(p, lds[256 + (16 * j + row) * 16 + ((4 * s + q) ^ row)], acc[j]);
      }
      wave_sync();
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < RT; ++j) sums[(wave * RT + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * 64; e += 64 * WAVES) {
      f32x4 v = sums[e];
#pragma unroll
      for (int i = 1; i < WAVES; ++i) v += sums[i * RT * 64 + e];
      const int l = e & 63, k2 = r0 + 16 * (e >> 6) + (l & 15);
      if (k2 >= a.rp) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int tk = 4 * (l >> 4) + c;
        if ((lanes >> tk) & 1)
          a.parts[((int64_t)blockIdx.y * a.m + t0 + tk) * a.rp + k2] = k2 < a.r ? v[c] * factor : 0.f;
      }
    }
  }
}

// Many tokens at ranks over 32, where the weights are the larger operand: a block takes 64 tokens, 16 a wave, and the
// waves share the weights, 128 columns at a time through LDS as above.
template <typename T, bool DROP, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES) void k_adapt_down_tiles(Down a, float factor) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int COLS = 128, RT = 4, BUF = (RT + WAVES) * 256;
  u32x4* lds = reinterpret_cast<u32x4*>(smem);  // [2][weights RT * 256, then 256 of each wave's tokens]
  const int lane = lane_id(), wave = threadIdx.x >> 6, row = lane & 15, q = lane >> 4;
  // (an XCD, every eighth block, takes the same ranges of the contraction for all tokens: its L2 holds their weights)
  const int split = blockIdx.x % a.splits;
  const int64_t t0 = (int64_t)(blockIdx.x / a.splits) * 64;
  const int r0 = blockIdx.y * (16 * RT);
  const int64_t kb = (int64_t)split * a.per;
  const int64_t ke = kb + a.per < a.K ? kb + a.per : a.K;
  const Philox g = DROP ? philox_of(a.drop.seed) : Philox{0u, 0u, 0u, 0u};
  const PhiloxMask mask = philox_mask_of(a.drop.threshold);

  // this lane's pieces: row 4 i + q of the wave's tokens, and of the weights every 16th row of the block
  int64_t prow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + 16 * wave + 4 * i + q;
    prow[i] = (t < a.m ? t : a.m - 1) * a.K;  // (a row past the last is not kept)
  }
  TileIds tile(a.ids, a.S, t0 + lane, t0 + lane < a.m);
  int adapter;
  uint64_t lanes;
  while (tile.next(adapter, lanes)) {
    const bool works = (lanes >> (16 * wave)) & 0xFFFFu;
    const T* w = (const T*)a.W + adapter * a.wstride;
    u32x4 x[4], y[RT];
    auto load = [&](int64_t k) {
      const int64_t at = k + 8 * row, left = a.K - at;
      if (works) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const T* p = (const T*)a.P + prow[i] + at;
          if (ALIGNED) x[i] = left > 0 ? *reinterpret_cast<const u32x4*>(p) : kZero4;  // (K is whole pieces)
          else x[i] = left >= 8 ? load_any(p) : load_some(p, left);
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        int r = r0 + (int)(threadIdx.x >> 4) + 16 * i;
        if (r >= a.r) r = a.r - 1;  // (its column is not kept)
        // (the rows of W are whole pieces, padded with zeros where P's are not)
        y[i] = left > 0 ? *reinterpret_cast<const u32x4*>(w + r * a.ldw + at) : kZero4;
      }
    };
    auto store = [&](int64_t k, int buf) {
      u32x4* to = lds + buf * BUF;
      if (works) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * i + q;
          if constexpr (DROP) {
            const u32x4 rnd = philox_block(g, (uint64_t)(prow[i] + k + 8 * row) / 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = philox_mask2(rnd[j], mask, x[i][j]);
          }
          to[(RT + wave) * 256 + r * 16 + (row ^ r)] = x[i];
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int r = (int)(threadIdx.x >> 4);
        to[i * 256 + r * 16 + (row ^ r)] = y[i];
      }
    };
    f32x4 acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int buf = 0;
    load(kb);
    __syncthreads();  // (the last adapter's operands are still read)
    store(kb, 0);
    __syncthreads();
    for (int64_t k = kb; k < ke; k += COLS) {
      const bool more = k + COLS < ke;
      if (more) load(k + COLS);
      if (works) {
        const u32x4* from = lds + buf * BUF;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const u32x4 p = from[(RT + wave) * 256 + row * 16 + ((4 * s + q) ^ row)];
#pragma unroll
          for (int j = 0; j < RT; ++j)
            acc[j] = mma<T>(p, from[j * 256 + row * 16 + ((4 * s + q) ^ row)], acc[j]);
        }
      }
      buf ^= 1;
      if (more) store(k + COLS, buf);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int k = r0 + 16 * j + row;
      if (k >= a.rp) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int tk = 16 * wave + 4 * q + c;
        if ((lanes >> tk) & 1)
          a.parts[((int64_t)split * a.m + t0 + tk) * a.rp + k] = k < a.r ? acc[j][c] * factor : 0.f;
      }
    }
  }
}

// the ranges' sums into the first one's place, in order
__global__ __launch_bounds__(256) void k_adapt_sum(float* parts, int64_t count, int splits) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  f32x4 t = *reinterpret_cast<const f32x4*>(parts + i);
#pragma unroll 4
  for (int s = 1; s < splits; ++s) t += *reinterpret_cast<const f32x4*>(parts + s * count + i);
  *reinterpret_cast<f32x4*>(parts + i) = t;
}

}  // namespace

// Ranges of the contraction: as many as bring the launch to 512 blocks, with at least one chunk for every wave of a
// block (or four chunks in turn, where the waves share them).
int down_splits(int64_t m, int64_t K, int r, int S, int64_t& per) {
  int64_t tiles = (m + 15) / 16, unit = 64, least = 64 * WAVES;
  int64_t adapters = S < m ? (S < 16 ? S : 16) : (m < 16 ? m : 16);
  if (m > kManyTokens) {
    if (r > kSharedRank) tiles = (m + 63) / 64;
    adapters = 1;
    unit = 128;
    least = 128 * WAVES;
  }
  int64_t want = 512 / (tiles * adapters);
  const int64_t most = (K + least - 1) / least;
  if (want > most) want = most;
  if (want < 1) want = 1;
  per = ((K + want - 1) / want + unit - 1) / unit * unit;
  return (int)((K + per - 1) / per);
}

hipError_t launch_down(Down& a, int dtype, hipStream_t s) {
  // the share that stays divides the sums: one multiplication per sum instead of one per value
  const float factor = a.drop.threshold ? a.drop.inv() : 1.f;
  auto go = [&](auto t, auto rt, auto drop, auto aligned) {
    typedef typename decltype(t)::type T;
    constexpr int RT = decltype(rt)::value;
    const int groups = (a.r + 16 * RT - 1) / (16 * RT);
    const int64_t tiles = (a.m + 15) / 16;
    const int most = a.S < 16 ? a.S : 16;
    int64_t Z = 1024 / (tiles * a.splits);
    if (Z > most) Z = most;
    if (Z < 1) Z = 1;
    if (a.m > kManyTokens && a.r > kSharedRank) {
      if constexpr (RT == 4)
        hipLaunchKernelGGL((k_adapt_down_tiles<T, decltype(drop)::value, decltype(aligned)::value>),
                           dim3((unsigned)((a.m + 63) / 64 * a.splits), (unsigned)groups), dim3(64 * WAVES),
                           2 * (4 + WAVES) * 4096, s, a, factor);
      return hipGetLastError();
    }
    if (a.m > kManyTokens) {
      if constexpr (RT == 4) return hipErrorNotSupported;  // (no such call comes here)
      const auto kern = k_adapt_down_lds<T, RT, decltype(drop)::value, decltype(aligned)::value>;
      constexpr size_t lds = WAVES * (1 + RT) * 4096;
      static const hipError_t ready = prepare_kernel((const void*)kern, lds);
      if (ready != hipSuccess) return ready;
      hipLaunchKernelGGL(kern, dim3((unsigned)tiles, (unsigned)a.splits, (unsigned)groups), dim3(64 * WAVES), lds, s, a,
                         factor);
      return hipGetLastError();
    }
    hipLaunchKernelGGL((k_adapt_down<T, RT, decltype(drop)::value, decltype(aligned)::value>),
                       dim3((unsigned)tiles, (unsigned)a.splits, (unsigned)(Z * groups)), dim3(64 * WAVES),
                       WAVES * RT * 64 * 16, s, a, (int)Z, factor);
    return hipGetLastError();
  };
  std::true_type yes;
  std::false_type no;
  auto with_ranks = [&](auto t, auto drop, auto aligned) {
    if (a.r <= 16) return go(t, std::integral_constant<int, 1>{}, drop, aligned);
    if (a.r <= 32) return go(t, std::integral_constant<int, 2>{}, drop, aligned);
    return go(t, std::integral_constant<int, 4>{}, drop, aligned);
  };
  auto with_rest = [&](auto t) {
    if (a.drop.threshold) return with_ranks(t, yes, yes);
    return a.K % 8 == 0 ? with_ranks(t, no, yes) : with_ranks(t, no, no);
  };
  hipError_t e = dtype == DT_F16 ? with_rest(dtype_of<DT_F16>{}) : with_rest(dtype_of<DT_BF16>{});
  // every wave of the next kernel reads the sums of its tokens: with several ranges they are added up once
  if (e == hipSuccess && a.m > kManyTokens && a.splits > 2) {
    const int64_t count = a.m * a.rp;
    hipLaunchKernelGGL(k_adapt_sum, dim3((unsigned)((count + 1023) / 1024)), dim3(256), 0, s, a.parts, count, a.splits);
    e = hipGetLastError();
    a.splits = 1;
  }
  return e;
}

}  // namespace adapt
}  // namespace skm
