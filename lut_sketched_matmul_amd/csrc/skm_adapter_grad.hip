// Gradients of the adapters' weights, dB_s = sum_t dy_t (scale_s h_t)^T and
// dA_s = sum_t dh_t D(x_t)^T over the tokens of adapter s (skm_adapter.h), and
// the calls that order all of the adapters' kernels.
//
// Positions. k_adapt_prepare lists every adapter's tokens in order, each list
// padded to whole steps of 32 positions (-1) and cut into chunks of at most
// `chunk` tokens. Without ids the list is the tokens themselves.
//
// k_adapt_grad: a block takes one chunk and 128 columns of dY or X; its waves
// take turns over the steps. The contraction runs over tokens, so a lane's
// operand is one column of eight tokens: it loads eight tokens' 16 bytes (16
// lanes: 256 consecutive bytes of a row) and turns the 8 x 8 values in registers,
// half an instruction a value. The other operand, the terms of h or dh, comes
// from k_adapt_terms in the order the lanes want it. An adapter of one chunk
// is written at once; the others' chunks are added up in order by
// k_adapt_reduce (deterministic, no atomics).
//
// 8192 tokens, 4096 -> 4096, rank 16, bf16 with dropout: 34 us for the 134 MB of dY and X (4 TB/s), bound by the
// vector ALU's share beside the loads (random numbers and turning: 40 % of its cycles) at two waves per SIMD; f16
// rows of 4095 values 39 us for 65 MB, their conversions and split lines more.
#include <type_traits>

#include "skm_adapter.h"
#include "skm_quant.h"

namespace skm {
namespace adapt {

namespace {

constexpr int STEP = 32;    // positions of a matrix instruction
constexpr int GTERMS = 3;   // bf16 terms of h and dh
constexpr int PLAN_THREADS = 1024;

struct Chunk {
  int32_t begin, end;  // positions, begin a multiple of STEP; none when end <= begin
  int32_t adapter;
  int32_t slot;        // where its sums go, -1 = the gradient itself
};
struct Owner {
  int32_t slot, count;  // an adapter's partial sums: first and how many (0 = none, 1 = written at once)
};

// ---- the adapters' tokens -----------------------------------------------------------

// exclusive sums over the block's threads (PLAN_THREADS of them); total in `all`
__device__ __forceinline__ int block_scan(int v, int* sh, int& all) {
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // (sh of an earlier call is still read)
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < PLAN_THREADS / 64; ++w) {
    if (w < wave) before += sh[w];
    all += sh[w];
  }
  return before + x - v;
}

__device__ __forceinline__ int chunks_of(int count, int chunk) { return (count + chunk - 1) / chunk; }

struct Plan {
  const int32_t* ids;
  int64_t m;
  int S, chunk, max_chunks, blocks;  // blocks: S, or 0 without a plan
  int32_t* order;
  Chunk* chunks;
  Owner* owners;
};
// Block `me` of S: counts all adapters' tokens, then writes its own list, chunks and owner. The last block marks the
// chunks nobody has. Sums over integers only: the order of the LDS atomics cannot show.
__device__ __forceinline__ void plan_block(const Plan& a, int me, int* hist, int* sh, int* mine) {
  const int32_t* __restrict__ ids = a.ids;
  const int64_t m = a.m;
  const int S = a.S, chunk = a.chunk, max_chunks = a.max_chunks, lane = lane_id();
  int32_t* order = a.order;
  Chunk* chunks = a.chunks;
  Owner* owners = a.owners;
  for (int i = threadIdx.x; i < S; i += PLAN_THREADS) hist[i] = 0;
  __syncthreads();
  for (int64_t t = threadIdx.x; t < (m + 63) / 64 * 64; t += PLAN_THREADS) {
    const int id = t < m ? ids[t] : -1;
    const bool in = id >= 0 && id < S;
    // a request's tokens stand together: one addition for a wave whose lanes agree
    const uint64_t live = __ballot(in);
    if (!live) continue;
    const int first = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(live));
    if (__ballot(in && id == first) == live) {
      if (lane == 0) atomicAdd(&hist[first], __builtin_popcountll(live));
    } else if (in) {
      atomicAdd(&hist[id], 1);
    }
  }
  __syncthreads();
  int pos = 0, nch = 0, nsl = 0;  // totals of the adapters before i
  for (int i0 = 0; i0 < S; i0 += PLAN_THREADS) {
    const int i = i0 + threadIdx.x;
    const int c = i < S ? hist[i] : 0, k = chunks_of(c, chunk);
    int all;
    const int p = pos + block_scan((c + STEP - 1) / STEP * STEP, sh, all);
    pos += all;
    const int q = nch + block_scan(k, sh, all);
    nch += all;
    const int z = nsl + block_scan(k > 1 ? k : 0, sh, all);
    nsl += all;
    if (i == me) {
      mine[0] = p;
      mine[1] = q;
      mine[2] = z;
    }
  }
  __syncthreads();
  const int begin = mine[0], count = hist[me], k = chunks_of(count, chunk);
  for (int i = threadIdx.x; i < k; i += PLAN_THREADS) {
    const int e = (i + 1) * chunk < count ? (i + 1) * chunk : count;
    chunks[mine[1] + i] = Chunk{begin + i * chunk, begin + e, me, k > 1 ? mine[2] + i : -1};
  }
  if (threadIdx.x == 0) owners[me] = Owner{mine[2], k};
  if (me == S - 1)
    for (int i = nch + threadIdx.x; i < max_chunks; i += PLAN_THREADS) chunks[i] = Chunk{0, 0, 0, -1};
  const int padded = (count + STEP - 1) / STEP * STEP;
  for (int i = count + threadIdx.x; i < padded; i += PLAN_THREADS) order[begin + i] = -1;
  if (!count) return;
  int done = 0;
  for (int64_t t0 = 0; t0 < m; t0 += PLAN_THREADS) {
    const int64_t t = t0 + threadIdx.x;
    const int is = t < m && ids[t] == me ? 1 : 0;
    int all;
    const int at = block_scan(is, sh, all);
    if (is) order[begin + done + at] = (int32_t)t;
    done += all;
  }
}

// B [S][n][r] -> [S][r][ld], zeros from n on: block i turns 64 rows of one adapter
struct Turn {
  const uint16_t* B;
  int64_t n, ld;
  int r;
  int64_t blocks;
  uint16_t* out;
};
__device__ __forceinline__ void turn_block(const Turn& a, int64_t block, uint16_t* tile) {
  const int64_t per = a.ld / 64, s = block / per, i0 = block % per * 64, n = a.n;
  const int r = a.r, ldt = r + 2;
  __syncthreads();  // (an earlier tile is still read)
  const uint16_t* b = a.B + (s * n + i0) * r;
  const int rows = (int)(n - i0 < 64 ? n - i0 : 64);
  for (int e = threadIdx.x; e < 64 * r; e += PLAN_THREADS) {
    const int i = e / r, k = e - i * r;
    tile[i * ldt + k] = i < rows ? b[e] : (uint16_t)0;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 64 * r; e += PLAN_THREADS) {
    const int k = e >> 6, i = e & 63;
    a.out[(s * r + k) * a.ld + i0 + i] = tile[i * ldt + k];
  }
}

// both, neither of which waits for the other: the first p.blocks blocks plan, the others turn
__global__ __launch_bounds__(PLAN_THREADS) void k_adapt_prepare(Plan p, Turn t) {
  extern __shared__ __align__(16) unsigned char smem[];  // S counters, or a tile of B
  __shared__ int sh[PLAN_THREADS / 64], mine[3];
  if ((int64_t)blockIdx.x < p.blocks) plan_block(p, blockIdx.x, (int*)smem, sh, mine);
  else
    for (int64_t b = (int64_t)blockIdx.x - p.blocks; b < t.blocks; b += gridDim.x - p.blocks)
      turn_block(t, b, (uint16_t*)smem);
}

// ---- operands --------------------------------------------------------------------

struct Terms {
  const float* parts;  // [splits][m][ld]
  int splits, ld;
  float factor;
  uint32_t* out;       // NULL = not wanted
};

// The terms of h (or dh) by position, as a matrix instruction's lanes want them: [step][term][16 ranks][lane][8
// positions] bf16, lane l rank l % 16 and positions 8 (l / 16) .. of the step's 32; zeros where there is no token or
// rank. A thread: two positions of one rank.
__global__ __launch_bounds__(256) void k_adapt_terms(Terms a, Terms b, const int32_t* __restrict__ ids,
                                                     const float* __restrict__ scale,
                                                     const int32_t* __restrict__ order, int64_t m, int64_t positions,
                                                     int r, int rp16, int S) {
  const Terms& t = blockIdx.y ? b : a;
  if (!t.out) return;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t step = e / (16 * rp16);
  if (step * STEP >= positions) return;
  const int in = (int)(e - step * (16 * rp16));
  const int rank = in % rp16, pair = in / rp16;  // neighbours read neighbouring ranks of a token
  float v[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t p = step * STEP + 2 * pair + j;
    const int64_t tk = order ? (p < positions ? order[p] : -1) : (p < m ? p : -1);
    v[j] = 0.f;
    if (tk >= 0 && tk < m && rank < r) {
      for (int i = 0; i < t.splits; ++i) v[j] += t.parts[((int64_t)i * m + tk) * t.ld + rank];
      const int id = ids ? ids[tk] : 0;
      // (a listed token has an adapter; positions behind the lists hold anything)
      v[j] *= scale && id >= 0 && id < S ? scale[id] * t.factor : t.factor;
    }
  }
#pragma unroll
  for (int k = 0; k < GTERMS; ++k) {
    const uint32_t w = pack2<bf16_t>(v[0], v[1]);
    t.out[((step * GTERMS + k) * rp16 + (rank & ~15)) * (STEP / 2) + ((rank & 15) + 16 * (pair >> 2)) * 4 + (pair & 3)] = w;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float u = unpack<bf16_t>(w, j);
      v[j] = __builtin_isfinite(u) ? v[j] - u : 0.f;
    }
  }
}

// ---- the products over tokens ----------------------------------------------------------

struct Grad {
  const void* P;        // dY or X, [m][N]
  int64_t N;
  const uint16_t* terms;
  float* out;           // dB [S][N][r] or dA [S][r][N]
  float* part;          // partial sums, one gradient each
  Dropout drop;
  int by_rank;          // dA: ranks are rows of the result
};
struct GradGrid {
  Grad b, a;            // dB, dA (columns 0 = not wanted)
  int64_t strips_b, strips;  // 128-column strips of dB, and of both
  const int32_t* order;
  const Chunk* chunks;  // NULL: chunk i is tokens [i chunk, (i + 1) chunk)
  int64_t m;
  int chunk, r, rp16, accumulate, single;  // single: without ids, one chunk in all
};

// a lane's eight tokens of a step, -1 past the chunk
__device__ __forceinline__ void load_tokens(const GradGrid& a, int p0, int end, int (&tk)[8]) {
  if (a.order) {
    // (whole steps are listed: both vectors are there)
    const int at = p0 < end ? p0 : 0;
    const u32x4 lo = reinterpret_cast<const u32x4*>(a.order + at)[0], hi = reinterpret_cast<const u32x4*>(a.order + at)[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) tk[i] = p0 + i < end ? (int)(i < 4 ? lo[i & 3] : hi[i & 3]) : -1;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) tk[i] = p0 + i < end ? p0 + i : -1;
  }
}
// their eight columns from col on, zeros where there is no token or column
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_rows(const Grad& g, int64_t col, const int (&tk)[8], u32x4 (&row)[8]) {
  if (ALIGNED || col + 8 <= g.N) {
    const int64_t c = col < g.N ? col : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const T* p = (const T*)g.P + (int64_t)(tk[i] < 0 ? 0 : tk[i]) * g.N + c;
      row[i] = ALIGNED ? *reinterpret_cast<const u32x4*>(p) : load_any(p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      row[i] = load_some((const T*)g.P + (int64_t)(tk[i] < 0 ? 0 : tk[i]) * g.N + col, g.N - col);
  }
}

// two bf16 terms of packed f16 values (exact together; an infinity's rest is NaN, and its sums are)
__device__ __forceinline__ void split_f16(u32x4 v, u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = unpack<half_t>(v[j], 0), b = unpack<half_t>(v[j], 1);
    hi[j] = pack2<bf16_t>(a, b);
    const float c = a - unpack<bf16_t>(hi[j], 0), d = b - unpack<bf16_t>(hi[j], 1);
    lo[j] = pack2<bf16_t>(c, d);
  }
}

template <typename T, int RT, bool ALIGNED>
__global__ __launch_bounds__(64 * WAVES) void k_adapt_grad(GradGrid a) {
  __shared__ __align__(16) f32x4 sums[WAVES][8][64];
  const int lane = lane_id(), wave = threadIdx.x >> 6, row = lane & 15, q = lane >> 4;
  const int64_t strip = (int64_t)blockIdx.x % a.strips, chunk_at = (int64_t)blockIdx.x / a.strips;
  const bool is_a = strip >= a.strips_b;
  const Grad& g = is_a ? a.a : a.b;
  const int64_t c0 = (strip - (is_a ? a.strips_b : 0)) * 128, col = c0 + 8 * row;
  const int r0 = (int)blockIdx.y * 16 * RT;
  Chunk ch;
  if (a.chunks) {
    ch = a.chunks[chunk_at];
  } else {
    const int64_t b = chunk_at * a.chunk, e = b + a.chunk;
    ch = Chunk{(int32_t)b, (int32_t)(e < a.m ? e : a.m), 0, a.single ? -1 : (int32_t)chunk_at};
  }
  if (ch.end <= ch.begin) return;
  const Philox rng = g.drop.threshold ? philox_of(g.drop.seed) : Philox{0u, 0u, 0u, 0u};

  f32x4 acc[RT][8];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[j][e] = f32x4{0.f, 0.f, 0.f, 0.f};
  const PhiloxMask mask = philox_mask_of(g.drop.threshold);

  // one step: its terms, the next step's rows and the tokens of the one behind that on their way, then the products
  constexpr int TURN = STEP * WAVES;
  auto step = [&](int p0, u32x4 (&x)[8], int (&tk)[8], u32x4 (&x_next)[8], int (&tk_next)[8]) {
    u32x4 h[GTERMS][RT];
    const uint16_t* tp = g.terms + (int64_t)(p0 / STEP) * (GTERMS * a.rp16 * STEP) + 8 * lane;
#pragma unroll
    for (int k = 0; k < GTERMS; ++k)
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int rank = r0 + 16 * j;  // (ranks past the last are not kept)
        h[k][j] = *reinterpret_cast<const u32x4*>(tp + (k * a.rp16 + (rank < a.rp16 ? rank : 0)) * STEP);
      }
    if (p0 + TURN < ch.end) load_rows<T, ALIGNED>(g, col, tk_next, x_next);
    if (p0 + STEP > ch.end) {  // (the last step of a chunk)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (tk[i] < 0) x[i] = kZero4;
    }
    if (ALIGNED && col >= g.N) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = kZero4;
    }
    if (g.drop.threshold) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const u32x4 rnd = philox_block(rng, (uint64_t)((int64_t)(tk[i] < 0 ? 0 : tk[i]) * g.N + col) / 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = philox_mask2(rnd[j], mask, x[i][j]);
      }
    }
    load_tokens(a, p0 + 2 * TURN + 8 * q, ch.end, tk);
    u32x4 y[8];
    turn8x8(x, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (__is_same(T, half_t)) {
        u32x4 hi, lo;
        split_f16(y[e], hi, lo);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          // smallest products first; lo times the third term is below 2^-24 of the whole
          acc[j][e] = mma<bf16_t>(h[1][j], lo, acc[j][e]);
          acc[j][e] = mma<bf16_t>(h[2][j], hi, acc[j][e]);
          acc[j][e] = mma<bf16_t>(h[0][j], lo, acc[j][e]);
          acc[j][e] = mma<bf16_t>(h[1][j], hi, acc[j][e]);
          acc[j][e] = mma<bf16_t>(h[0][j], hi, acc[j][e]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          acc[j][e] = mma<bf16_t>(h[2][j], y[e], acc[j][e]);
          acc[j][e] = mma<bf16_t>(h[1][j], y[e], acc[j][e]);
          acc[j][e] = mma<bf16_t>(h[0][j], y[e], acc[j][e]);
        }
      }
    }
  };
  int t0[8], t1[8];
  u32x4 x0[8], x1[8];
  int p0 = ch.begin + STEP * wave;
  load_tokens(a, p0 + 8 * q, ch.end, t0);
  load_tokens(a, p0 + TURN + 8 * q, ch.end, t1);
  if (p0 < ch.end) load_rows<T, ALIGNED>(g, col, t0, x0);
  if constexpr (RT == 1 && ALIGNED) {
    while (p0 < ch.end) {
      step(p0, x0, t0, x1, t1);
      p0 += TURN;
      if (p0 >= ch.end) break;
      step(p0, x1, t1, x0, t0);
      p0 += TURN;
    }
  } else {  // (two copies of the step do not fit the registers, or leave them for two waves per SIMD instead of three)
    for (; p0 < ch.end; p0 += TURN) {
      step(p0, x0, t0, x1, t1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = t0[i];
        x0[i] = x1[i];
        t0[i] = t1[i];
        t1[i] = t;
      }
    }
  }

  const int64_t size = (int64_t)a.r * g.N;
  float* out = ch.slot < 0 ? g.out + ch.adapter * size : g.part + ch.slot * size;
  const bool add = ch.slot < 0 && a.accumulate;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[wave][e][lane] = acc[j][e];
    __syncthreads();
    // lane l of instruction e: column c0 + 8 (l % 16) + e, ranks 4 (l / 16) .. + 3
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int v = (int)threadIdx.x + 256 * i;
      int e, l;
      if (g.by_rank) {  // eight threads: the eight columns of a lane
        e = v & 7;
        l = v >> 3;
      } else {          // a column's ranks: four threads
        l = ((v >> 5) & 15) | (v & 3) << 4;
        e = (v >> 2) & 7;
      }
      f32x4 t = sums[0][e][l];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) t += sums[w][e][l];
      const int64_t c = c0 + 8 * (l & 15) + e;
      const int k0 = r0 + 16 * j + 4 * (l >> 4);
      if (c < g.N) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (k0 + x < a.r) {
            float* o = out + (g.by_rank ? (k0 + x) * g.N + c : c * a.r + k0 + x);
            *o = add ? *o + t[x] : t[x];
          }
      }
    }
  }
}

// adapters with no chunk (zeros) or with several (their sums, in order)
__global__ __launch_bounds__(256) void k_adapt_reduce(Grad b, Grad a, const Owner* __restrict__ owners, int only_count,
                                                      int r, int accumulate) {
  const Grad& g = blockIdx.z ? a : b;
  const int64_t size = (int64_t)r * g.N;
  const int s = blockIdx.y;
  const Owner o = owners ? owners[s] : Owner{0, s ? 0 : only_count};  // (without ids all tokens are adapter 0's)
  if (!g.out || o.count == 1) return;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= size) return;
  const float* p = g.part + (int64_t)o.slot * size + i;
  float* out = g.out + s * size + i;
  if (size % 4 == 0) {
    f32x4 t = accumulate ? *reinterpret_cast<const f32x4*>(out) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < o.count; ++k) t += *reinterpret_cast<const f32x4*>(p + k * size);
    *reinterpret_cast<f32x4*>(out) = t;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < size) {
        float t = accumulate ? out[j] : 0.f;
        for (int k = 0; k < o.count; ++k) t += p[k * size + j];
        out[j] = t;
      }
  }
}

// ---- sizes ---------------------------------------------------------------------------

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// what a backward call needs, and where it lies in the workspace
struct Layout {
  int64_t per, ldt, positions, max_chunks, slots;
  int splits, rp, rp16, chunk;
  size_t turned, parts, order, chunks, owners, terms_h, terms_dh, part_b, part_a, bytes;
};

Layout layout_of(const AdapterArgs& a, bool need_dx, bool need_da, bool need_db) {
  Layout l{};
  const int64_t S = a.ids ? a.S : 1;
  l.rp = padded_rank(a.r);
  l.rp16 = (a.r + 15) / 16 * 16;
  l.ldt = (a.n + 63) / 64 * 64;
  l.splits = down_splits(a.m, a.n, a.r, (int)S, l.per);
  // Chunks: as long as the launch keeps 512 blocks, since every chunk costs a partial gradient (written and read
  // again); whole turns of the block's waves. (8192 tokens, 4096 -> 4096, rank 16: 34 us, with 1024 blocks 36.5.)
  // Several adapters' tokens do not come in whole chunks, and shorter ones even that out (4001 tokens, 4096 -> 4095,
  // rank 12, 5 adapters: 1024 blocks 39 us, 512 54).
  const int64_t strips = (need_db ? (a.n + 127) / 128 : 0) + (need_da ? (a.d + 127) / 128 : 0);
  int64_t chunk = a.m * strips / (a.ids ? 1024 : 512);
  const int64_t least = 16 * a.r;  // a partial gradient is then at most a quarter of the data read
  if (chunk < least) chunk = least;
  if (chunk > 4096) chunk = 4096;
  l.chunk = (int)((chunk + STEP * WAVES - 1) / (STEP * WAVES) * (STEP * WAVES));
  const int64_t some = S < a.m ? S : a.m;  // adapters that can have tokens
  if (a.ids) {
    l.positions = a.m + some * (STEP - 1);
    l.max_chunks = a.m / l.chunk + some;
    l.slots = 2 * a.m / l.chunk;  // (an adapter of k > 1 chunks has more than k / 2 chunks of tokens)
  } else {
    l.positions = a.m;
    l.max_chunks = (a.m + l.chunk - 1) / l.chunk;
    l.slots = l.max_chunks > 1 ? l.max_chunks : 0;
  }
  l.positions = (l.positions + STEP - 1) / STEP * STEP;
  size_t at = 0;
  auto take = [&](bool want, size_t bytes) {
    const size_t o = at;
    if (want) at += up256(bytes);
    return o;
  };
  const bool dh = need_dx || need_da, grads = need_da || need_db;
  l.turned = take(dh, (size_t)(S * a.r * l.ldt) * 2);
  l.parts = take(dh, (size_t)l.splits * a.m * l.rp * 4);
  l.order = take(grads && a.ids, (size_t)l.positions * 4);
  l.chunks = take(grads && a.ids, (size_t)l.max_chunks * sizeof(Chunk));
  l.owners = take(grads && a.ids, (size_t)S * sizeof(Owner));
  const size_t terms = (size_t)l.positions * l.rp16 * GTERMS * 2;
  l.terms_h = take(need_db, terms);
  l.terms_dh = take(need_da, terms);
  l.part_b = take(need_db, (size_t)(l.slots * a.r * a.n) * 4);
  l.part_a = take(need_da, (size_t)(l.slots * a.r * a.d) * 4);
  l.bytes = at;
  return l;
}

struct FwdLayout {
  int64_t per;
  int splits, rp;
  size_t bytes;
};
FwdLayout fwd_layout(const AdapterArgs& a) {
  FwdLayout l{};
  l.rp = padded_rank(a.r);
  l.splits = down_splits(a.m, a.d, a.r, a.ids ? a.S : 1, l.per);
  l.bytes = up256((size_t)l.splits * a.m * l.rp * 4);
  return l;
}

}  // namespace

}  // namespace adapt

using namespace adapt;

size_t adapter_fwd_bytes(const AdapterArgs& a) { return few_tokens(a) ? 0 : fwd_layout(a).bytes; }

hipError_t launch_adapter_fwd(const AdapterArgs& a, const void* base, void* Y, float* H, void* ws, hipStream_t s) {
  if (few_tokens(a)) return launch_few(a, base, Y, H, s);
  const FwdLayout l = fwd_layout(a);
  const int S = a.ids ? a.S : 1;
  Down dn{a.X, a.A, a.d, (int64_t)a.r * a.d, a.m, a.d, l.per, a.r, l.rp, S, l.splits, a.ids, a.drop, (float*)ws};
  const hipError_t e = launch_down(dn, a.dtype, s);
  if (e != hipSuccess) return e;
  Up up{(const float*)ws, dn.splits, l.rp, a.r, S, a.B, a.m, a.n, a.ids, a.scale, 1.f, base, Y, H, Dropout{0, nullptr}};
  return launch_up(up, a.dtype, false, s);
}

size_t adapter_bwd_bytes(const AdapterArgs& a, bool need_dx, bool need_da, bool need_db) {
  return layout_of(a, need_dx, need_da, need_db).bytes;
}

hipError_t launch_adapter_bwd(const AdapterArgs& a, const void* dY, const float* H, const float* base_dx, void* dX,
                              float* dA, float* dB, int accumulate, void* ws, hipStream_t s) {
  const Layout l = layout_of(a, dX != nullptr, dA != nullptr, dB != nullptr);
  const int S = a.ids ? a.S : 1;
  unsigned char* w = (unsigned char*)ws;
  float* parts = (float*)(w + l.parts);
  int32_t* order = a.ids ? (int32_t*)(w + l.order) : nullptr;
  Chunk* chunks = a.ids ? (Chunk*)(w + l.chunks) : nullptr;
  Owner* owners = a.ids ? (Owner*)(w + l.owners) : nullptr;
  hipError_t e = hipSuccess;
  int splits = l.splits;  // left to add up
  const bool dh = dX || dA, plan = (dA || dB) && a.ids;
  uint16_t* turned = (uint16_t*)(w + l.turned);
  if (dh || plan) {
    const Plan p{a.ids, a.m, S, l.chunk, (int)l.max_chunks, plan ? S : 0, order, chunks, owners};
    const Turn t{(const uint16_t*)a.B, a.n, l.ldt, a.r, dh ? l.ldt / 64 * S : 0, turned};
    const int64_t most = int64_t(1) << 20, turns = t.blocks < most ? t.blocks : most;
    const size_t counters = plan ? (size_t)S * 4 : 0, tile = dh ? (size_t)64 * (a.r + 2) * 2 : 0;
    hipLaunchKernelGGL(k_adapt_prepare, dim3((unsigned)(p.blocks + turns)), dim3(PLAN_THREADS),
                       counters > tile ? counters : tile, s, p, t);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (dh) {
    Down dn{dY,  turned, l.ldt, a.r * l.ldt, a.m, a.n, l.per, a.r, l.rp, S, l.splits, a.ids, Dropout{0, nullptr},
            parts};
    if ((e = launch_down(dn, a.dtype, s)) != hipSuccess) return e;
    splits = dn.splits;
  }
  if (dA || dB) {
    const float inv = a.drop.threshold ? a.drop.inv() : 1.f;
    const Terms th{H, 1, a.r, 1.f, dB ? (uint32_t*)(w + l.terms_h) : nullptr};
    const Terms td{parts, splits, l.rp, inv, dA ? (uint32_t*)(w + l.terms_dh) : nullptr};
    const int64_t threads = l.positions / STEP * 16 * l.rp16;
    hipLaunchKernelGGL(k_adapt_terms, dim3((unsigned)((threads + 255) / 256), 2), dim3(256), 0, s, th, td, a.ids,
                       a.scale, order, a.m, l.positions, a.r, l.rp16, S);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const Grad gb{dY, a.n, (const uint16_t*)(w + l.terms_h), dB, (float*)(w + l.part_b), Dropout{0, nullptr}, 0};
    const Grad ga{a.X, a.d, (const uint16_t*)(w + l.terms_dh), dA, (float*)(w + l.part_a), a.drop, 1};
    const int64_t sb = dB ? (a.n + 127) / 128 : 0, sa = dA ? (a.d + 127) / 128 : 0;
    const int64_t blocks = (sb + sa) * l.max_chunks;
    const GradGrid g{gb, ga, sb, sb + sa, order, chunks, a.m,
                     l.chunk, a.r, l.rp16, accumulate, l.max_chunks == 1};
    auto go = [&](auto t, auto rt, auto al) {
      constexpr int RT = decltype(rt)::value;
      hipLaunchKernelGGL((k_adapt_grad<typename decltype(t)::type, RT, decltype(al)::value>),
                         dim3((unsigned)blocks, (unsigned)((l.rp16 + 16 * RT - 1) / (16 * RT))),
                         dim3(64 * WAVES), 0, s, g);
      return hipGetLastError();
    };
    auto with_ranks = [&](auto t, auto al) {
      if (a.r <= 16) return go(t, std::integral_constant<int, 1>{}, al);
      if (a.r <= 32) return go(t, std::integral_constant<int, 2>{}, al);
      return go(t, std::integral_constant<int, 4>{}, al);
    };
    // (X's rows are whole vectors always; dY's when n is a multiple of 8)
    auto with_rows = [&](auto t) {
      return a.n % 8 == 0 || !dB ? with_ranks(t, std::true_type{}) : with_ranks(t, std::false_type{});
    };
    e = a.dtype == DT_F16 ? with_rows(dtype_of<DT_F16>{}) : with_rows(dtype_of<DT_BF16>{});
    if (e != hipSuccess) return e;
    // (one adapter's single chunk is everything, and is written already)
    if (a.ids || l.max_chunks > 1 || a.S > 1) {
      const int64_t most = (dB && dA ? (a.n > a.d ? a.n : a.d) : (dB ? a.n : a.d)) * a.r;
      hipLaunchKernelGGL(k_adapt_reduce, dim3((unsigned)((most + 1023) / 1024), (unsigned)a.S, 2), dim3(256), 0, s, gb, ga,
                         owners, (int)l.max_chunks, a.r, accumulate);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  if (dX) {
    const float inv = a.drop.threshold ? a.drop.inv() : 1.f;
    Up up{parts, splits, l.rp, a.r, S, a.A, a.m, a.d, a.ids, a.scale, inv, base_dx, dX, nullptr, a.drop};
    if ((e = launch_up(up, a.dtype, true, s)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace skm
