// Cross entropy of a sketched head: the small kernels around the tiles (token
// list, merge of the statistics, gather of X, dX's last sum) and the host
// side that cuts the vocabulary into pieces. The mathematics is in skm_xent.h.
#include "skm_gemm_common.h"
#include "skm_quant.h"
#include "skm_xent.h"

namespace skm {

namespace {

constexpr int XENT_BN = 256;  // vocabulary rows of a tile

// ---- the ranges of dX ---------------------------------------------------------------
// The ranges of dX's tiles for the tokens there are. Up to half a round of 256
// tiles: as many equal ranges as make rounds of 256 blocks times 64-row steps
// per block least (at least 4 steps each, two rounds at the most, `cap` token
// rows of sums for all ranges). Otherwise the tiles past whole rounds, R of them
// (R <= 224), are cut in two: with q = ceil(R / (256 - R)) short ranges for each
// CU left over, a long range takes q steps of q + 1. (3 / 4 of 4096 tokens, 4096
// columns: 192 tiles, 192 ranges of 3 / 4 of the steps beside 64 CUs with three
// of 1 / 4 each.) Thread t looks at t + 1 equal ranges.
struct DxShape {
  int32_t nb, steps;  // column tiles, steps of the first piece
  int64_t cap;
};
constexpr int DX_CUT_STEPS = 32;  // fewest steps of a tile cut in two: none of 7 / 8 and 1 / 8 of them is empty
__device__ __forceinline__ DxPlan dx_plan(int32_t count, const DxShape& q, unsigned long long* slot) {
  const uint32_t tiles = (uint32_t)(count + 255) / 256u * (uint32_t)q.nb, steps = (uint32_t)q.steps;
  if (tiles > 128u || count == 0) {  // block-uniform
    const uint32_t R = tiles % 256u;
    if (R == 0 || R > 224u || q.steps < DX_CUT_STEPS || q.cap < 2 * (int64_t)count) return {(int32_t)tiles, 1, 1, 1};
    const int32_t c = (int32_t)(255u / (256u - R));  // ceil(R / (256 - R))
    return {(int32_t)(tiles - R), 2, c, c + 1};
  }
  const uint32_t t = threadIdx.x + 1;
  unsigned long long best = ~0ull;
  if (t == 1 || (4 * t <= steps && tiles * t <= 512u && count * (int64_t)t <= q.cap))
    best = ((unsigned long long)((tiles * t + 255u) / 256u) * ((steps + t - 1) / t)) << 10 | t;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const unsigned long long v = __shfl_xor(best, o, 64);
    best = v < best ? v : best;
  }
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) best = slot[w] < best ? slot[w] : best;
  const uint32_t c = (uint32_t)best & 1023u, len = (steps + c - 1) / c, k = (steps + len - 1) / len;
  return {0, (int32_t)k, 1, (int32_t)k};
}

// ---- the list of tokens that have a target -----------------------------------------
// One block (the list is one scan over m targets, 8192 per round).
// rows[c] = token of listed row c, in token order. Forward: loss and lse of the
// others are zeroed. Backward: pos[t] = listed row of token t or -1, and the
// power of two that puts the largest finite |dloss| 2^e (e from zexp, NULL = 0)
// into [2^14, 2^15) (1 when there is none).
__device__ __forceinline__ uint32_t larger_finite(uint32_t top, float f) {
  const uint32_t a = __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu;
  return a < 0x7F800000u && a > top ? a : top;
}
template <bool BWD>
__global__ void __launch_bounds__(1024) k_xent_index(const int64_t* __restrict__ targets, int64_t ignore, int64_t m,
                                                     const float* __restrict__ dloss,
                                                     const int32_t* __restrict__ zexp, XentHead* __restrict__ head,
                                                     int32_t* __restrict__ rows, int32_t* __restrict__ pos,
                                                     DxShape dx, float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ int32_t before[129];  // listed tokens of a round in front of wave w's k-th 64: [16 k + w]
  __shared__ unsigned long long slot[16];
  __shared__ uint32_t wmax[16];
  const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
  int32_t base = 0;
  uint32_t top = 0u;
  for (int64_t r0 = 0; r0 < m; r0 += 8192) {
    unsigned long long on[8];
    float f[8] = {};
    int32_t z[8] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = r0 + 1024 * k + t;
      bool mine = false;
      if (i < m) {
        mine = targets[i] != ignore;
        if constexpr (BWD) {
          f[k] = dloss[i];
          if (zexp) z[k] = zexp[i];
        }
      }
      on[k] = __ballot(mine);
      if (lane == 0) before[16 * k + wave] = __popcll(on[k]);
    }
    __syncthreads();
    if (wave == 0) {
      const int32_t a = before[2 * lane], s = a + before[2 * lane + 1];
      int32_t scan = s;  // inclusive over the wave
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int32_t v = __shfl_up(scan, o, 64);
        if (lane >= o) scan += v;
      }
      before[2 * lane] = scan - s;
      before[2 * lane + 1] = scan - s + a;
      if (lane == 63) before[128] = scan;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = r0 + 1024 * k + t;
      if (i >= m) continue;
      const bool mine = (on[k] >> lane) & 1u;
      const int32_t c = base + before[16 * k + wave] + __popcll(on[k] & ((1ull << lane) - 1u));
      if (mine) rows[c] = (int32_t)i;
      if constexpr (BWD) {
        pos[i] = mine ? c : -1;
        if (mine) top = larger_finite(top, f[k] * pow2f(z[k]));
      } else if (!mine) {
        loss[i] = 0.0f;
        lse[i] = 0.0f;
      }
    }
    base += before[128];
    __syncthreads();  // (the next round writes before)
  }
  if constexpr (BWD) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const uint32_t v = (uint32_t)__shfl_xor((int)top, o, 64);
      top = top > v ? top : v;
    }
    if (lane == 0) wmax[wave] = top;
    __syncthreads();
  }
  DxPlan plan{0, 1, 1, 1};
  if constexpr (BWD)
    if (dx.nb > 0) plan = dx_plan(base, dx, slot);
  if (t == 0) {
    head->count = base;
    head->dx = plan;
    if constexpr (BWD) {
      for (int w = 0; w < 16; ++w) top = top > wmax[w] ? top : wmax[w];
      const int e = scale_exp(top);
      head->scale = pow2f(e);
      head->inv_scale = pow2f(-e);
    }
  }
}

// ---- the listed rows for the streaming logit tiles --------------------------------------
// Xp[c] = X[rows[c]] in the tables' dtype TL, every 8 columns in the K order of
// mm::dequant8_b4. SC (bf16 with f16 tables): prescaled by 2^-e of the row, e
// written to rexp[token] (skm_common.h). One block per row; the second read of
// a scaled row comes from the caches.
template <typename TX, typename TL>
__global__ void __launch_bounds__(256) k_xent_rows(const TX* __restrict__ X, const int32_t* __restrict__ rows,
                                                   const XentHead* __restrict__ head, int64_t d, TL* __restrict__ Xp,
                                                   int32_t* __restrict__ rexp) {
  constexpr bool SC = scaled_pair(__is_same(TX, bf16_t), __is_same(TL, half_t));
  __shared__ uint32_t top[4];
  const int64_t c = blockIdx.x;
  if (c >= head->count) return;
  const int64_t t = rows[c];
  const u32x4* src = reinterpret_cast<const u32x4*>(X + t * d);
  u32x4* dst = reinterpret_cast<u32x4*>(Xp + c * d);
  float scale = 1.0f;
  if constexpr (SC) {
    uint32_t mx = 0u;
    for (int64_t j = threadIdx.x; j < d / 8; j += 256) {
      const uint32_t a = absmax8_bf16(src[j]);
      mx = mx > a ? mx : a;
    }
    mx = wave_max_to_lane63(mx);
    if ((threadIdx.x & 63) == 63) top[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) mx = w == 0 || top[w] > mx ? top[w] : mx;
    const int e = row_exp_of(mx);
    scale = pow2f(-e);
    if (threadIdx.x == 0) rexp[t] = e;
  }
  for (int64_t j = threadIdx.x; j < d / 8; j += 256) {
    if constexpr (SC) dst[j] = mm::cvt_quad_perm_scaled(src[j], scale);
    else dst[j] = mm::cvt_quad_perm<TX, TL>(src[j]);
  }
}
hipError_t xent_rows(const XentGemm& g, void* Xp, int32_t* rexp, hipStream_t s) {
  const dim3 grid((unsigned)g.p.m);
  if (g.x_dtype == DT_F16)
    hipLaunchKernelGGL((k_xent_rows<half_t, half_t>), grid, dim3(256), 0, s, (const half_t*)g.X, g.rows, g.head, g.p.d,
                       (half_t*)Xp, rexp);
  else if (g.lut_dtype == DT_F16)
    hipLaunchKernelGGL((k_xent_rows<bf16_t, half_t>), grid, dim3(256), 0, s, (const bf16_t*)g.X, g.rows, g.head,
                       g.p.d, (half_t*)Xp, rexp);
  else
    hipLaunchKernelGGL((k_xent_rows<bf16_t, bf16_t>), grid, dim3(256), 0, s, (const bf16_t*)g.X, g.rows, g.head,
                       g.p.d, (bf16_t*)Xp, rexp);
  return hipGetLastError();
}

// ---- forward: merge of the blocks' (max, sum) pairs ------------------------------------
// 16 listed tokens per block, 16 threads each over the vocabulary blocks.
__global__ void __launch_bounds__(256) k_xent_merge(const float2* __restrict__ part, int64_t stride, int nvb,
                                                    const XentHead* __restrict__ head,
                                                    const int32_t* __restrict__ rows,
                                                    const int64_t* __restrict__ targets, int64_t V,
                                                    const float* __restrict__ tlogit, float* __restrict__ loss,
                                                    float* __restrict__ lse) {
  __shared__ float sm[16][16], ss[16][16];
  const int tk = (int)(threadIdx.x & 15), sl = (int)(threadIdx.x >> 4);
  const int64_t c = (int64_t)blockIdx.x * 16 + tk;
  const int count = head->count;
  if ((int64_t)blockIdx.x * 16 >= count) return;  // block-uniform
  float mx = -__builtin_inff(), sum = 0.0f;
  if (c < count) {
    for (int v = sl; v < nvb; v += 16) {
      const float2 p = part[(int64_t)v * stride + c];
      const float nm = __builtin_fmaxf(mx, p.x);
      const float ref = nm == -__builtin_inff() ? 0.0f : nm;
      sum = sum * __expf(mx - ref) + p.y * __expf(p.x - ref);
      mx = nm;
    }
  }
  sm[sl][tk] = mx;
  ss[sl][tk] = sum;
  __syncthreads();
  if (sl != 0 || c >= count) return;
  mx = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < 16; ++i) mx = __builtin_fmaxf(mx, sm[i][tk]);
  const float ref = mx == -__builtin_inff() ? 0.0f : mx;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += ss[i][tk] * __expf(sm[i][tk] - ref);
  const float l = ref + logf(sum);
  const int64_t t = rows[c];
  const int64_t target = targets[t];
  lse[t] = l;
  loss[t] = target >= 0 && target < V ? l - tlogit[c] : __builtin_nanf("");
}

// The same for few tokens: a block per token over its [blocks] pairs, ignored
// tokens included.
__global__ void __launch_bounds__(1024) k_xent_merge_few(const float2* __restrict__ part, int64_t blocks,
                                                         const int64_t* __restrict__ targets, int64_t ignore,
                                                         int64_t V, const float* __restrict__ tlogit,
                                                         float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float sm[16], ss[16];
  const int64_t t = blockIdx.x;
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  float mx = -__builtin_inff(), sum = 0.0f;
  auto add = [&](float m2, float s2) {
    const float nm = __builtin_fmaxf(mx, m2);
    const float ref = nm == -__builtin_inff() ? 0.0f : nm;
    sum = sum * __expf(mx - ref) + s2 * __expf(m2 - ref);
    mx = nm;
  };
  for (int64_t v = threadIdx.x; v < blocks; v += 1024) {
    const float2 p = part[t * blocks + v];
    add(p.x, p.y);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const float m2 = __shfl_xor(mx, o, 64), s2 = __shfl_xor(sum, o, 64);
    add(m2, s2);
  }
  if (lane == 0) {
    sm[wave] = mx;
    ss[wave] = sum;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  mx = sm[0];
  sum = ss[0];
  for (int w = 1; w < 16; ++w) add(sm[w], ss[w]);
  const int64_t target = targets[t];
  const bool live = target != ignore;
  const float l = (mx == -__builtin_inff() ? 0.0f : mx) + logf(sum);
  lse[t] = live ? l : 0.0f;
  loss[t] = !live ? 0.0f : (target >= 0 && target < V ? l - tlogit[t] : __builtin_nanf(""));
}

// mean of the scored losses and every token's weight in it: one block, a chain
// per thread, then the 1024 sums as a tree
__global__ void __launch_bounds__(1024) k_xent_mean(const float* __restrict__ loss, const int64_t* __restrict__ targets,
                                                    int64_t ignore, int64_t m, float* __restrict__ mean,
                                                    float* __restrict__ weight) {
  __shared__ float ssum[16];
  __shared__ int32_t scnt[16];
  float sum = 0.0f;
  int32_t cnt = 0;
  for (int64_t t = threadIdx.x; t < m; t += 1024) {
    const bool on = targets[t] != ignore;
    sum += on ? loss[t] : 0.0f;
    cnt += on ? 1 : 0;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    sum += __shfl_xor(sum, o, 64);
    cnt += __shfl_xor(cnt, o, 64);
  }
  if ((threadIdx.x & 63) == 0) {
    ssum[threadIdx.x >> 6] = sum;
    scnt[threadIdx.x >> 6] = cnt;
  }
  __syncthreads();
  sum = 0.0f;
  cnt = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    sum += ssum[w];
    cnt += scnt[w];
  }
  const float wt = cnt > 0 ? 1.0f / (float)cnt : 0.0f;
  if (threadIdx.x == 0) *mean = cnt > 0 ? sum / (float)cnt : 0.0f;
  for (int64_t t = threadIdx.x; t < m; t += 1024) weight[t] = targets[t] != ignore ? wt : 0.0f;
}

// ---- backward --------------------------------------------------------------------------

// Xc[c] = X[rows[c]] in f16 for the listed tokens (bf16 rows prescaled by 2^-e,
// e = zexp: their largest value then lies in [2^14, 2^15)), zeros up to the next
// multiple of 32 (whole steps of the table gradient's tiles); 16 bytes per thread
// and round
template <typename TX>
__global__ void __launch_bounds__(256) k_xent_gather(const TX* __restrict__ X, const int32_t* __restrict__ rows,
                                                     const int32_t* __restrict__ zexp,
                                                     const XentHead* __restrict__ head, int64_t d,
                                                     half_t* __restrict__ Xc) {
  const int64_t c = blockIdx.x;
  const int count = head->count;
  if (c >= ((int64_t)count + 31) / 32 * 32) return;
  const bool live = c < count;
  const int64_t t = live ? rows[c] : 0;
  float scale = 1.0f;
  if constexpr (__is_same(TX, bf16_t)) scale = live ? pow2f(-zexp[t]) : 1.0f;
  const u32x4* src = reinterpret_cast<const u32x4*>(X + t * d);
  u32x4* dst = reinterpret_cast<u32x4*>(Xc + c * d);
  for (int64_t j = threadIdx.x; j < d / 8; j += 256) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (live) {
      v = src[j];
      if constexpr (__is_same(TX, bf16_t)) v = mm::cvt_quad_scaled(v, scale);
    }
    dst[j] = v;
  }
}

// dX[t] = (sum of the ranges' dX of t's listed row + what rounding took from the
// target's term, times the target's weights), scaled back; zeros for an ignored
// token. f16 operands (TL) carry the token's scale (dloss given) or dLUT's, bf16
// ones none. A block sums 2048 / lanes columns, 8 per thread, `lanes` threads
// taking every lanes-th range each: a few rows have up to 256 ranges, which one
// thread would wait for one by one.
template <int B, typename TX, typename TL>
__global__ void __launch_bounds__(256) k_xent_dx_out(const float* __restrict__ acc, int lanes,
                                                     const int32_t* __restrict__ pos,
                                                     const XentHead* __restrict__ head,
                                                     const float* __restrict__ dloss,
                                                     const float* __restrict__ rest,
                                                     const int64_t* __restrict__ targets,
                                                     const uint8_t* __restrict__ idx_packed,
                                                     const TL* __restrict__ lut, int64_t V, int64_t d, int gpr,
                                                     TX* __restrict__ dX) {
  constexpr int K = 1 << B;
  __shared__ float part[8][256];  // [column of a thread's eight][thread]
  const int64_t t = blockIdx.x;
  const int64_t c = pos[t];
  const int64_t target = targets[t];
  const int chunks = 256 / lanes, lane = (int)threadIdx.x / chunks;
  const int64_t j = 8 * ((int64_t)blockIdx.y * chunks + (int)threadIdx.x % chunks);
  const bool fix = c >= 0 && target >= 0 && target < V && j < d && lane == 0;
  // the 8 indices of columns j .. j + 7 are B bytes (one group: its width is a multiple of 32)
  uint32_t w = 0u;
  float r = 0.0f;
  if (fix) {
    const uint8_t* row = idx_packed + target * (d * B / 8) + j / 8 * B;
#pragma unroll
    for (int q = 0; q < B; ++q) w |= (uint32_t)row[q] << (8 * q);
    r = rest[c];
  }
  float v[8] = {};
  if (c >= 0 && j < d) {
    const float* src = acc + c * d + j;
    const int64_t count = head->count, part_stride = count * d;
    const DxPlan q = head->dx;
    const int ranges = j / 256 * ((count + 255) / 256) + c / 256 >= q.cut_from ? q.ranges : 1;
    int k = lane;
    for (; k + 3 * lanes < ranges; k += 4 * lanes) {
      float a[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) load8<float>(src + (k + u * lanes) * part_stride, a[u]);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += (a[0][q] + a[1][q]) + (a[2][q] + a[3][q]);
    }
    for (; k < ranges; k += lanes) {
      float a[8];
      load8<float>(src + k * part_stride, a);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += a[q];
    }
  }
  if (lanes > 1) {  // block-uniform
#pragma unroll
    for (int q = 0; q < 8; ++q) part[q][threadIdx.x] = v[q];
    __syncthreads();
    if (lane > 0) return;
    for (int k = 1; k < lanes; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += part[q][k * chunks + threadIdx.x];
  }
  if (j >= d) return;
  if (fix) {
    const TL* g = lut + (target * gpr + (uint32_t)j / (uint32_t)(d / gpr)) * K;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = __builtin_fmaf(r, to_f32(g[(w >> (B * q)) & (K - 1)]), v[q]);
  }
  if constexpr (!__is_same(TL, bf16_t)) {
    const float back = !dloss ? head->inv_scale : (c >= 0 ? pow2f(-xent_token_exp(dloss[t])) : 0.0f);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= back;
  }
  store8<TX>(dX + t * d + j, v);
}

struct DxOut {
  const float* acc;
  int ranges;
  const int32_t* pos;
  const XentHead* head;
  const float* dloss;  // dX's operand is scaled token by token; NULL = as dLUT's
  const float* rest;
};
template <typename TX, typename TL>
hipError_t dx_out_t(const XentArgs& a, const DxOut& o, void* dX, hipStream_t s) {
  const Problem& p = a.p;
  // two or more of the most ranges per lane, and at most 2048 blocks' worth of threads
  int lanes = 1;
  while (lanes < 32 && lanes * 2 <= o.ranges && p.m * p.d * lanes < 2048 * 2048) lanes *= 2;
  const int64_t cols = 2048 / lanes;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)p.m, (unsigned)((p.d + cols - 1) / cols)), dim3(256), 0, s, o.acc,
                       lanes, o.pos, o.head, o.dloss, o.rest, a.targets, a.idx, (const TL*)a.lut, p.n, p.d, p.gpr,
                       (TX*)dX);
    return hipGetLastError();
  };
  if (p.b == 2) return go(k_xent_dx_out<2, TX, TL>);
  if (p.b == 3) return go(k_xent_dx_out<3, TX, TL>);
  return go(k_xent_dx_out<4, TX, TL>);
}
hipError_t dx_out(const XentArgs& a, const DxOut& o, void* dX, hipStream_t s) {
  if (a.x_dtype == DT_F16) return dx_out_t<half_t, half_t>(a, o, dX, s);
  if (a.lut_dtype == DT_F16) return dx_out_t<bf16_t, half_t>(a, o, dX, s);
  return dx_out_t<bf16_t, bf16_t>(a, o, dX, s);
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

bool mixed(int x_dtype, int lut_dtype) { return scaled_pair(x_dtype == DT_BF16, lut_dtype == DT_F16); }

// ---- workspace layouts -----------------------------------------------------------------
struct FwdPlan {
  bool few;
  int64_t blocks;                          // vocabulary blocks of the statistics
  bool streams;                            // listed rows copied for the streaming tiles
  size_t rows, rexp, part, tlogit, xp, bytes;  // byte offsets (the head is at 0)
};
FwdPlan fwd_plan(const Problem& p, int x_dtype, int lut_dtype) {
  FwdPlan f;
  f.few = xent_few(p);
  f.streams = !f.few && xent_streams(p);
  f.blocks = f.few ? (p.n + 15) / 16 : (p.n + XENT_BN - 1) / XENT_BN;
  size_t o = 256;
  f.rows = o;
  o += up256((size_t)p.m * 4);
  f.rexp = o;
  if (mixed(x_dtype, lut_dtype)) o += up256((size_t)p.m * 4);
  f.part = o;
  o += up256((size_t)f.blocks * (size_t)p.m * 8);
  f.tlogit = o;
  o += up256((size_t)p.m * 4);
  f.xp = o;
  if (f.streams) o += up256((size_t)p.m * (size_t)p.d * 2);
  f.bytes = o;
  return f;
}

struct BwdPlan {
  int64_t cap;         // listed rows, rounded up to 32
  int64_t P;           // vocabulary rows per piece
  int64_t slots;       // dX sums of m tokens in the workspace (the most ranges when all have a target, or 2)
  int64_t dx_blocks;   // the most blocks of dX's ranges for any number of listed tokens
  DxShape dx;
  bool few, streams;
  bool own;            // dX's operand is a form of its own
  bool rexps, zexps;   // bf16 rows in f16: exponents of the logits' operand rows, of dLUT's
  size_t rows, pos, rexp, zexp, hi, lo, dxv, rest, acc, xc, xp, part, bytes;
};

// The pieces: dZ of a piece takes 2 bytes per (token, word) and form, and is
// written once and read by two products; 256 MB of it stays in the memory-side
// cache, and more rows per piece only save re-reading dX's fp32 sums. A piece
// has at least one tile of words, which is more than that from 175 000 tokens
// (three forms) to 524 000 (one) on.
constexpr size_t XENT_PIECE_BYTES = size_t(256) << 20;

BwdPlan bwd_plan(const Problem& p, int x_dtype, int lut_dtype, bool need_dx, bool need_dlut) {
  BwdPlan f;
  f.own = x_dtype == DT_BF16;
  const bool has_hi = need_dlut || !f.own, has_dxv = need_dx && f.own;
  f.rexps = mixed(x_dtype, lut_dtype);
  f.zexps = x_dtype == DT_BF16 && need_dlut;
  const int forms = (has_hi ? 1 : 0) + (need_dlut ? 1 : 0) + (has_dxv ? 1 : 0);
  f.few = xent_few(p);
  f.streams = !f.few && xent_streams(p);
  f.cap = (p.m + 31) / 32 * 32;
  int64_t P = (int64_t)(XENT_PIECE_BYTES / (size_t)(f.cap * 2 * forms)) / XENT_BN * XENT_BN;
  if (P < XENT_BN) P = XENT_BN;
  const int64_t pieces = (p.n + P - 1) / P;
  P = ((p.n + pieces - 1) / pieces + XENT_BN - 1) / XENT_BN * XENT_BN;
  f.P = P;
  const int64_t n1 = p.n < P ? p.n : P;
  const int64_t nb = (p.d + 255) / 256, tiles = (p.m + 255) / 256 * nb;
  f.slots = dx_ranges(Problem{p.m, n1, p.d, p.b, p.gpr}).count;
  if (f.slots < 2) f.slots = 2;
  f.dx = DxShape{need_dx ? (int32_t)nb : 0, (int32_t)((n1 + 63) / 64), f.slots * p.m};
  const int64_t most = f.dx.steps < 8 ? 1 : f.dx.steps / 4;  // equal ranges
  f.dx_blocks = tiles <= 128 ? (tiles * most < 512 ? tiles * most : 512) : (tiles + 224 > 512 ? tiles + 224 : 512);
  size_t o = 256;
  auto take = [&](bool on, size_t bytes) {
    const size_t at = o;
    if (on) o += up256(bytes);
    return at;
  };
  const size_t dz = (size_t)f.cap * (size_t)((n1 + 7) / 8 * 8) * 2;
  f.rows = take(true, (size_t)p.m * 4);
  f.pos = take(true, (size_t)p.m * 4);
  f.rexp = take(f.rexps, (size_t)p.m * 4);
  f.zexp = take(f.zexps, (size_t)p.m * 4);
  f.rest = take(need_dx, (size_t)p.m * 4);
  f.hi = take(has_hi, dz);
  f.lo = take(need_dlut, dz);
  f.dxv = take(has_dxv, dz);
  f.acc = take(need_dx, (size_t)f.slots * (size_t)p.m * (size_t)p.d * 4);
  f.xc = take(need_dlut, (size_t)f.cap * (size_t)p.d * 2);
  size_t part = 0;
  for (int64_t v0 = 0; v0 < p.n; v0 += P) {  // (the last piece may split differently)
    if (v0 > 0 && v0 + P < p.n) continue;
    const Problem q{f.cap, p.n - v0 < P ? p.n - v0 : P, p.d, p.b, p.gpr};
    const size_t b = dlut_partial_bytes(q);
    part = b > part ? b : part;
  }
  f.part = take(need_dlut, part);
  f.xp = take(f.streams, (size_t)p.m * (size_t)p.d * 2);
  f.bytes = o;
  return f;
}

template <typename T> T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

}  // namespace

// Whether the decode kernel, 16 tokens per block, beats the 256 x 256 tiles: it
// dequantises for every 16 tokens, about 0.4 + 0.00014 d ns per word and group of
// them with the chip full; the tiles take about 10 + 0.021 d us per round of 256
// blocks however few of a block's tokens exist. Both sides measured for b = 2, 3
// and 4 and 1 to 8 groups (statistics, us, decode against tiles): 32000 words of
// 4096 columns, 16 / 32 / 64 tokens 36 / 64 / 117 against 105; 16000 of 2048, 32
// / 64 / 160 tokens 31 / 54 / 121 against 59; 4000 of 4096, 64 / 160 / 300 / 500
// tokens 23 / 45 / 77 / 124 against 100; 2048 of 1024, 160 / 500 tokens 19 / 46
// against 38. The gradient takes the same rule (its dZ has to come from the
// logits that lse came from); there the decode's two-byte stores bring the
// crossover forward a little, at most 8 % of a call (dX alone, us): 32000 of
// 4096, 16 / 32 / 48 / 64 tokens 115 / 145 / 176 / 207 against 172 to 180; 16000
// of 2048, 32 / 64 / 160 tokens 70 / 100 / 184 against 88 / 93 / 103; 4000 of
// 4096, 160 / 300 / 500 tokens 78 / 120 / 175 against 134 / 141 / 146.
bool xent_few(const Problem& p) {
  const int64_t groups = (p.m + 15) / 16, tiles = (p.m + 255) / 256 * ((p.n + XENT_BN - 1) / XENT_BN);
  const double decode = (double)(groups * p.n) * (0.4e-3 + 0.14e-6 * (double)p.d);
  const int64_t blocks = ((p.n + 15) / 16 + 7) / 8 * 8 * groups;
  return decode <= (double)((tiles + 255) / 256) * (10.0 + 0.021 * (double)p.d) &&
         // (a launch has fewer than 2^32 threads: 512 per block here, 1024 per token in k_xent_merge_few)
         blocks <= (int64_t(1) << 22) && p.m < (int64_t(1) << 22) &&
         decode_supported(Problem{p.m < 16 ? p.m : 16, p.n, p.d, p.b, p.gpr});
}

// 32 KB of a block's LDS: two blocks or more share a CU then (8 tokens of 4096
// columns, 32000 words: 53 us staged, 36 us from memory; 64 of 2048, 16000
// words: 85 against 54)
bool xent_decode_stages(const Problem& p) { return (p.m < 16 ? p.m : 16) * p.d <= 16384; }

size_t xent_fwd_bytes(const Problem& p, int x_dtype, int lut_dtype) { return fwd_plan(p, x_dtype, lut_dtype).bytes; }

hipError_t launch_xent_fwd(const XentArgs& a, float* loss, float* lse, void* ws, hipStream_t s) {
  const Problem& p = a.p;
  const FwdPlan f = fwd_plan(p, a.x_dtype, a.lut_dtype);
  XentHead* head = at<XentHead>(ws, 0);
  int32_t* rows = at<int32_t>(ws, f.rows);
  int32_t* rexp = mixed(a.x_dtype, a.lut_dtype) ? at<int32_t>(ws, f.rexp) : nullptr;
  float2* part = at<float2>(ws, f.part);
  float* tlogit = at<float>(ws, f.tlogit);
  void* xp = f.streams ? at<void>(ws, f.xp) : nullptr;
  const XentGemm g{a.X, a.x_dtype, a.idx, a.lut, a.lut_dtype, p, rows, head, a.targets, rexp, 0, xp};
  hipError_t e = hipSuccess;
  if (f.few) {
    if (rexp && !xent_decode_stages(p)) e = launch_row_exp(a.X, p.m, p.d, rexp, s);
    if (e == hipSuccess) e = xent_few_stats(g, part, f.blocks, tlogit, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_xent_merge_few, dim3((unsigned)p.m), dim3(1024), 0, s, part, f.blocks, a.targets, a.ignore,
                       p.n, tlogit, loss, lse);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_xent_index<false>, dim3(1), dim3(1024), 0, s, a.targets, a.ignore, p.m, nullptr, nullptr, head,
                     rows, nullptr, DxShape{}, loss, lse);
  e = hipGetLastError();
  if (e == hipSuccess && f.streams) e = xent_rows(g, xp, rexp, s);
  else if (e == hipSuccess && rexp) e = launch_row_exp(a.X, p.m, p.d, rexp, s);
  if (e != hipSuccess) return e;
  e = xent_stats(g, part, p.m, tlogit, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_xent_merge, dim3((unsigned)((p.m + 15) / 16)), dim3(256), 0, s, part, p.m,
                     (int)f.blocks, head, rows, a.targets, p.n, tlogit, loss, lse);
  return hipGetLastError();
}

hipError_t launch_xent_mean(const float* loss, const int64_t* targets, int64_t ignore, int64_t m, float* mean,
                            float* weight, hipStream_t s) {
  hipLaunchKernelGGL(k_xent_mean, dim3(1), dim3(1024), 0, s, loss, targets, ignore, m, mean, weight);
  return hipGetLastError();
}

size_t xent_bwd_bytes(const Problem& p, int x_dtype, int lut_dtype, bool need_dx, bool need_dlut) {
  return bwd_plan(p, x_dtype, lut_dtype, need_dx, need_dlut).bytes;
}

hipError_t launch_xent_bwd(const XentArgs& a, const float* lse, const float* dloss, void* dX, float* dLUT,
                           int accumulate, void* ws, hipStream_t s) {
  const Problem& p = a.p;
  const BwdPlan f = bwd_plan(p, a.x_dtype, a.lut_dtype, dX != nullptr, dLUT != nullptr);
  XentHead* head = at<XentHead>(ws, 0);
  int32_t* rows = at<int32_t>(ws, f.rows);
  int32_t* pos = at<int32_t>(ws, f.pos);
  int32_t* rexp = f.rexps ? at<int32_t>(ws, f.rexp) : nullptr;
  // dLUT's operands: bf16 rows of X are scaled by 2^-e, their rows of dZ by 2^e
  int32_t* zexp = f.zexps ? at<int32_t>(ws, f.zexp) : nullptr;
  float* acc = dX ? at<float>(ws, f.acc) : nullptr;
  float* rest = dX ? at<float>(ws, f.rest) : nullptr;
  void* hi = dLUT || !f.own ? at<void>(ws, f.hi) : nullptr;
  void* lo = dLUT ? at<void>(ws, f.lo) : nullptr;
  void* dxv = dX && f.own ? at<void>(ws, f.dxv) : nullptr;
  void* xc = dLUT ? at<void>(ws, f.xc) : nullptr;
  void* xp = f.streams ? at<void>(ws, f.xp) : nullptr;
  hipError_t e = hipSuccess;
  // (xent_rows and the staging decode find the logits' exponents themselves)
  int32_t* find = f.streams || (f.few && xent_decode_stages(p)) ? nullptr : rexp;
  if (find || zexp) e = launch_row_exp(a.X, p.m, p.d, find, s, zexp);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_xent_index<true>, dim3(1), dim3(1024), 0, s, a.targets, a.ignore, p.m, dloss, zexp, head, rows,
                     pos, f.dx, nullptr, nullptr);
  e = hipGetLastError();
  XentGemm g{a.X, a.x_dtype, a.idx, a.lut, a.lut_dtype, p, rows, head, a.targets, rexp, 0, xp};
  if (e == hipSuccess && f.streams) e = xent_rows(g, xp, rexp, s);
  if (e == hipSuccess && dLUT) {
    if (a.x_dtype == DT_F16)
      hipLaunchKernelGGL(k_xent_gather<half_t>, dim3((unsigned)f.cap), dim3(256), 0, s, (const half_t*)a.X, rows, zexp,
                         head, p.d, (half_t*)xc);
    else
      hipLaunchKernelGGL(k_xent_gather<bf16_t>, dim3((unsigned)f.cap), dim3(256), 0, s, (const bf16_t*)a.X, rows, zexp,
                         head, p.d, (half_t*)xc);
    e = hipGetLastError();
  }
  const int es = 2;  // bytes of a table entry (16-bit pairs only)
  for (int64_t v0 = 0; v0 < p.n && e == hipSuccess; v0 += f.P) {
    const int64_t n = p.n - v0 < f.P ? p.n - v0 : f.P;
    const Problem q{p.m, n, p.d, p.b, p.gpr};
    const uint8_t* idx = a.idx + v0 * p.row_bytes();
    const void* lut = static_cast<const char*>(a.lut) + v0 * p.gpr * p.k() * es;
    const int64_t ld = (n + 7) / 8 * 8;
    g.idx = idx;
    g.lut = lut;
    g.p = q;
    g.v0 = v0;
    const XentGradOut out{lse, dloss, p.n, ld, hi, lo, dxv, zexp, rest};
    e = f.few ? xent_few_grad(g, out, pos, s) : xent_grad(g, out, s);
    if (e == hipSuccess && dX) {
      // every range of the first piece is written; later pieces add to some or all
      e = launch_dx_piece(f.own ? dxv : hi, a.lut_dtype, idx, lut, a.lut_dtype, q, acc, nullptr, &head->count, ld,
                          v0 > 0, {}, &head->dx, f.dx_blocks, s);
    }
    if (e == hipSuccess && dLUT) {
      const Problem qc{f.cap, n, p.d, p.b, p.gpr};
      e = launch_dlut_piece(hi, lo, xc, DT_F16, idx, qc, dLUT + v0 * p.gpr * p.k(), accumulate,
                            at<float>(ws, f.part), {&head->count, ld, &head->inv_scale, nullptr}, s);
    }
  }
  if (e != hipSuccess || !dX) return e;
  return dx_out(a, {acc, (int)f.slots, pos, head, f.own || !dLUT ? dloss : nullptr, rest}, dX, s);
}

}  // namespace skm
