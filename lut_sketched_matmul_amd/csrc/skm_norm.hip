// Layer norm and root-mean-square norm of the rows of X [m][d], forward and
// backward (the norm in front of a sketched layer).
//
//   layer: mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r
//   rms:   mu = 0,       r = 1 / sqrt(mean(x^2) + eps),        xh = x r
//   y  = xh w + b
//   dx = r (g - xh mean(g xh) - [layer] mean(g)),  g = dy w
//   dw = sum_rows dy xh,   db = sum_rows dy
//
// All arithmetic is fp32; means are quotients, rounded once. (As products with
// a rounded 1 / d, the mean of 7 times 1000 was 1000.0001 and y of that row 0.02
// instead of 0.) A row is read once and stays in registers: TPR threads of E = 8
// NCH elements each, so the variance is taken from the centred values (no
// cancellation) without a second read. Rows of whole 8-column chunks (AL) move 8
// consecutive columns per lane; other widths take the same kernels with column
// j TPR + t in element j of thread t.
//
// Backward: each block walks rows blockIdx, blockIdx + grid, ... and keeps its
// columns' dw and db sums in registers, the next row's loads in flight while a
// row is worked on; the block's sums go to the workspace and k_norm_reduce adds
// them per column in block order (deterministic, no atomics).
//
// Bound by memory from a few hundred rows on, by launch latency below. 8192 x
// 4096 bf16: forward with its checkpoint 30 us (5.6 TB/s), layer backward with
// fp32 dY 46 + 5 us (6.2 TB/s; a large copy reaches 5.15 to 6.2). 777 x 1001: 7 + 4 us;
// one row of 4096: 2.8 us. A forward that walks rows like the backward, or that
// fetches its next row early, measured the same.
#include <type_traits>

#include "skm_launch.h"
#include "skm_quant.h"

namespace skm {

namespace {

// column of element j (0..7) of chunk c of thread t
template <bool AL, int TPR>
__device__ __forceinline__ int col_of(int t, int c, int j) {
  return AL ? (c * TPR + t) * 8 + j : (c * 8 + j) * TPR + t;
}

// the thread's elements of a row as fp32, 0 past the row's end
template <typename T, bool AL, int TPR, int NCH>
__device__ __forceinline__ void load_row(const T* row, int d, int t, float (&v)[NCH][8]) {
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if constexpr (AL) {
      const int j0 = col_of<AL, TPR>(t, c, 0);
      if (j0 < d) {
        load8<T>(row + j0, v[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = col_of<AL, TPR>(t, c, j);
        v[c][j] = col < d ? to_f32(row[col]) : 0.0f;
      }
    }
  }
}

// a row as loaded: the conversion to fp32 waits until the row is worked on
template <typename T, bool AL, int NCH> struct RawRow {
  static constexpr int Q = __is_same(T, float) ? 2 : 1;
  u32x4 v[AL ? NCH * Q : 1];
  T e[AL ? 1 : NCH * 8];
};
template <typename T, bool AL, int TPR, int NCH>
__device__ __forceinline__ void load_raw(const T* row, int d, int t, RawRow<T, AL, NCH>& r) {
  typedef RawRow<T, AL, NCH> R;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if constexpr (AL) {
      const int j0 = col_of<AL, TPR>(t, c, 0);
#pragma unroll
      for (int q = 0; q < R::Q; ++q)
        r.v[c * R::Q + q] = j0 < d ? reinterpret_cast<const u32x4*>(row + j0)[q] : u32x4{0u, 0u, 0u, 0u};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = col_of<AL, TPR>(t, c, j);
        r.e[c * 8 + j] = col < d ? row[col] : from_f32<T>(0.0f);
      }
    }
  }
}
template <typename T, bool AL, int NCH>
__device__ __forceinline__ void from_raw(const RawRow<T, AL, NCH>& r, float (&v)[NCH][8]) {
  typedef RawRow<T, AL, NCH> R;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if constexpr (AL) {
      load8<T>(reinterpret_cast<const T*>(&r.v[c * R::Q]), v[c]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = to_f32(r.e[c * 8 + j]);
    }
  }
}
// the same for a checkpoint's row (AL only), `row` values from its start
template <int NCH> struct RawCodes {
  u32x2 v[NCH];
  uint32_t s[NCH];
};
template <int TPR, int NCH>
__device__ __forceinline__ void load_codes(const int8_t* codes, const uint8_t* scales, int64_t row, int d, int t,
                                           RawCodes<NCH>& o) {
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int j0 = col_of<true, TPR>(t, c, 0);
    const bool in = j0 < d;
    o.v[c] = in ? *reinterpret_cast<const u32x2*>(codes + row + j0) : u32x2{0u, 0u};
    o.s[c] = in ? scales[(row + j0) >> 5] : 1u;
  }
}

template <typename T, bool AL, int TPR, int NCH>
__device__ __forceinline__ void store_row(T* row, int d, int t, const float (&v)[NCH][8]) {
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if constexpr (AL) {
      const int j0 = col_of<AL, TPR>(t, c, 0);
      if (j0 < d) store8<T>(row + j0, v[c]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = col_of<AL, TPR>(t, c, j);
        if (col < d) row[col] = from_f32<T>(v[c][j]);
      }
    }
  }
}

// chunk c of a weight or bias row (fp32 or T; NULL gives `fill`). One assignment per
// element: with the three sources in branches of their own the compiler merged
// their stores and kept the array in scratch memory (8192 rows of 4096 columns
// forward: 6 KB of scratch written per row, 28.6 us instead of 22.6).
template <typename T, bool AL, int TPR>
__device__ __forceinline__ void load_param(const void* p, int p_f32, int d, int t, int c, float fill, float (&v)[8]) {
  const bool f = __is_same(T, float) || p_f32;
  const char* base = static_cast<const char*>(p);
  if constexpr (AL) {
    const int j0 = col_of<AL, TPR>(t, c, 0);
    const bool in = p && j0 < d;
    const u32x4* q = reinterpret_cast<const u32x4*>(base + (int64_t)j0 * (f ? 4 : 2));
    const u32x4 z = {0u, 0u, 0u, 0u};
    const u32x4 a = in ? q[0] : z, b = in && f ? q[1] : z;
    const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x = j < 4 ? fa[j & 3] : fb[j & 3];
      if constexpr (!__is_same(T, float)) {
        const uint32_t w = a[j >> 1];
        const float h = to_f32(__builtin_bit_cast(T, (uint16_t)(j & 1 ? w >> 16 : w & 0xFFFFu)));
        x = f ? x : h;
      }
      v[j] = p ? x : fill;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<AL, TPR>(t, c, j);
      const bool in = p && col < d;
      float x = in && f ? reinterpret_cast<const float*>(base)[col] : 0.0f;
      if constexpr (!__is_same(T, float)) {
        const float h = in && !f ? to_f32(reinterpret_cast<const T*>(base)[col]) : 0.0f;
        x = f ? x : h;
      }
      v[j] = p ? x : fill;
    }
  }
}

// sums of a and b over the TPR threads of a row (every thread gets them);
// `red` holds 2 floats per wave of the block. Block-uniform when TPR > 64.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int w = (int)(threadIdx.x >> 6);
    __syncthreads();  // the previous sums have been read
    if ((threadIdx.x & 63) == 0) {
      red[2 * w] = a;
      red[2 * w + 1] = b;
    }
    __syncthreads();
    a = 0.0f;
    b = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      a += red[2 * i];
      b += red[2 * i + 1];
    }
  }
}

// s / d rounded once, given 1 / d rounded (Markstein): the remainder of the
// product is exact in an fma and corrects its last bit. d is an integer of at
// most 17 bits, never the all-ones significand that the method leaves out. The
// same as a division in a third of its instructions: 4096 x 20000 forward 135 us,
// with divisions 141 (all waves of the CU's one block wait for them), with the
// products alone 133.
__device__ __forceinline__ float quotient(float s, float d, float inv_d) {
  const float q = s * inv_d;
  const float m = __builtin_fmaf(__builtin_fmaf(-q, d, s), inv_d, q);
  return __builtin_fabsf(q) < __builtin_inff() ? m : q;
}

template <typename T, bool AL, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
k_norm_fwd(const T* __restrict__ X, const void* __restrict__ w, const void* __restrict__ bias, int p_f32, int64_t m,
           int d, int layer, float eps, T* __restrict__ Y, float* __restrict__ mean, float* __restrict__ rstd,
           int8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[2 * (TPR / 64)];
  const int t = (int)(threadIdx.x % TPR);
  const int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (r >= m) return;  // uniform over the row's threads (the whole block when TPR > 64)
  float x[NCH][8];
  load_row<T, AL, TPR, NCH>(X + r * d, d, t, x);
  const float fd = (float)d, inv_d = 1.0f / fd;
  float mu = 0.0f, z = 0.0f;
  if (layer) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) mu += x[c][j];
    row_sum2<TPR>(mu, z, red);
    mu = quotient(mu, fd, inv_d);
  }
  float var = 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[c][j] = col_of<AL, TPR>(t, c, j) < d ? x[c][j] - mu : 0.0f;
      var = __builtin_fmaf(x[c][j], x[c][j], var);
    }
  z = 0.0f;
  row_sum2<TPR>(var, z, red);
  const float rs = 1.0f / sqrtf(quotient(var, fd, inv_d) + eps);
  if (t == 0) {
    rstd[r] = rs;
    if (mean) mean[r] = mu;
  }
  // the weights of all chunks together, of longer rows one chunk at a time (fewer
  // registers: 4096 x 16384 62 -> 52 us, 4096 x 20000 520 -> 160 us)
  constexpr int STEP = NCH <= 2 ? NCH : 1;
#pragma unroll
  for (int c0 = 0; c0 < NCH; c0 += STEP) {
    float p[STEP][8];
#pragma unroll
    for (int c = 0; c < STEP; ++c) load_param<T, AL, TPR>(w, p_f32, d, t, c0 + c, 1.0f, p[c]);
#pragma unroll
    for (int c = 0; c < STEP; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[c0 + c][j] = x[c0 + c][j] * rs * p[c][j];
    if (bias) {
#pragma unroll
      for (int c = 0; c < STEP; ++c) load_param<T, AL, TPR>(bias, p_f32, d, t, c0 + c, 0.0f, p[c]);
#pragma unroll
      for (int c = 0; c < STEP; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[c0 + c][j] += p[c][j];
    }
  }
  if (!AL || !codes) {
    store_row<T, AL, TPR, NCH>(Y + r * d, d, t, x);
    return;
  }
  if constexpr (AL) {  // d is a multiple of 32: the four lanes of a block are in range together
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j0 = col_of<AL, TPR>(t, c, 0);
      if (j0 >= d) continue;
      // the checkpoint is of Y as stored
      u32x4 y[sizeof(T) / 2];
      store8<T>(reinterpret_cast<T*>(y), x[c]);
#pragma unroll
      for (int q = 0; q < (int)sizeof(T) / 2; ++q) reinterpret_cast<u32x4*>(Y + r * d + j0)[q] = y[q];
      uint32_t s;
      *reinterpret_cast<u32x2*>(codes + r * d + j0) = ckpt_of<T>(y, s);
      if ((t & 3) == 0) scales[(r * d + j0) >> 5] = (uint8_t)s;
    }
  }
}

// DYF: dY is fp32 (else T); CK: X is a checkpoint. (At least two waves per SIMD:
// with one, 4096 x 8192 took 50 us instead of 44.)
template <typename T, bool AL, int TPR, int NCH, bool DYF, bool CK>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, AL && TPR == 256 ? 2 : 1)
k_norm_bwd(const void* __restrict__ dY, const T* __restrict__ X, const int8_t* __restrict__ codes,
           const uint8_t* __restrict__ scales, const void* __restrict__ w, int p_f32, const float* __restrict__ mean,
           const float* __restrict__ rstd, int64_t m, int d, T* __restrict__ dX, float* __restrict__ part_w,
           float* __restrict__ part_b) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  typedef std::conditional_t<DYF, float, T> TY;
  __shared__ float red[2 * (TPR / 64)];
  const int t = (int)(threadIdx.x % TPR);
  const float fd = (float)d, inv_d = 1.0f / fd;
  float p[NCH][8], aw[NCH][8], ab[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[c][j] = ab[c][j] = 0.0f;
  RawRow<TY, AL, NCH> rg;
  RawRow<T, AL, NCH> rx;
  RawCodes<NCH> rc;
  float mu = 0.0f, rs = 0.0f;
  auto load = [&](int64_t r) {
    load_raw<TY, AL, TPR, NCH>((const TY*)dY + r * d, d, t, rg);
    if constexpr (CK) load_codes<TPR, NCH>(codes, scales, r * d, d, t, rc);
    else load_raw<T, AL, TPR, NCH>(X + r * d, d, t, rx);
    mu = mean ? mean[r] : 0.0f;
    rs = rstd[r];
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (r < m) load(r);
#pragma unroll
  for (int c = 0; c < NCH; ++c) load_param<T, AL, TPR>(w, p_f32, d, t, c, 1.0f, p[c]);
  for (; r < m; r += step) {
    float x[NCH][8], g[NCH][8];
    from_raw<TY, AL, NCH>(rg, g);
    if constexpr (CK) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) ckpt_unpack8(rc.v[c], rc.s[c], x[c]);
    } else {
      from_raw<T, AL, NCH>(rx, x);
    }
    const float m0 = mu, r0 = rs;
    if (r + step < m) load(r + step);
    float s1 = 0.0f, s2 = 0.0f;  // sums of g xh and of g, g = dy w
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (x[c][j] - m0) * r0;  // (past the row's end dy is 0)
        aw[c][j] = __builtin_fmaf(g[c][j], xh, aw[c][j]);
        ab[c][j] += g[c][j];
        g[c][j] *= p[c][j];
        x[c][j] = xh;
        s1 = __builtin_fmaf(g[c][j], xh, s1);
        s2 += g[c][j];
      }
    if (dX) {
      row_sum2<TPR>(s1, s2, red);
      s1 = quotient(s1, fd, inv_d);
      s2 = mean ? quotient(s2, fd, inv_d) : 0.0f;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[c][j] = r0 * (g[c][j] - s2 - x[c][j] * s1);
      store_row<T, AL, TPR, NCH>(dX + r * d, d, t, x);
    }
  }
  // the block's sums: with several rows at a time, those of the row slots in order
  auto put = [&](float* part, float (&a)[NCH][8]) {
    if constexpr (RPB > 1) {
      __shared__ float slots[RPB - 1][NCH * 8][64];
      const int k = (int)(threadIdx.x >> 6);
      __syncthreads();
      if (k > 0) {
#pragma unroll
        for (int e = 0; e < NCH * 8; ++e) slots[k - 1][e][t] = a[e >> 3][e & 7];
      }
      __syncthreads();
      if (k > 0) return;
#pragma unroll
      for (int i = 0; i < RPB - 1; ++i)
#pragma unroll
        for (int e = 0; e < NCH * 8; ++e) a[e >> 3][e & 7] += slots[i][e][t];
    }
    store_row<float, AL, TPR, NCH>(part + (int64_t)blockIdx.x * d, d, t, a);
  };
  if (part_w) put(part_w, aw);
  if (part_b) put(part_b, ab);
}

// Rows of more than 16384 columns: a thread's columns and their sums do not fit
// its registers (in scratch memory 4096 x 20000 took 3.5 ms). dX reads its row
// twice, the second time from the caches; dw and db come from a pass by columns.

// x and g = dy of 8 columns of chunk c of row r, as fp32
template <typename T, bool AL, int TPR, bool DYF, bool CK>
__device__ __forceinline__ void load_pair(const void* dY, const T* X, const int8_t* codes, const uint8_t* scales,
                                          int64_t r, int d, int t, int c, float (&x)[1][8], float (&g)[1][8]) {
  typedef std::conditional_t<DYF, float, T> TY;
  const int base = c * 8 * TPR;
  load_row<TY, AL, TPR, 1>((const TY*)dY + r * d + base, d - base, t, g);
  if constexpr (CK) {
    RawCodes<1> q;
    load_codes<TPR, 1>(codes + base, scales + base / 32, r * d, d - base, t, q);
    ckpt_unpack8(q.v[0], q.s[0], x[0]);
  } else {
    load_row<T, AL, TPR, 1>(X + r * d + base, d - base, t, x);
  }
}

template <typename T, bool AL, bool DYF, bool CK>
__global__ void __launch_bounds__(1024)
k_norm_bwd_wide(const void* __restrict__ dY, const T* __restrict__ X, const int8_t* __restrict__ codes,
                const uint8_t* __restrict__ scales, const void* __restrict__ w, int p_f32,
                const float* __restrict__ mean, const float* __restrict__ rstd, int64_t m, int d,
                T* __restrict__ dX) {
  constexpr int TPR = 1024;
  __shared__ float red[2 * (TPR / 64)];
  const int t = (int)threadIdx.x, chunks = (d + 8 * TPR - 1) / (8 * TPR);
  const float fd = (float)d, inv_d = 1.0f / fd;
  for (int64_t r = blockIdx.x; r < m; r += gridDim.x) {
    const float mu = mean ? mean[r] : 0.0f, rs = rstd[r];
    float s1 = 0.0f, s2 = 0.0f;  // sums of g xh and of g, g = dy w
    for (int c = 0; c < chunks; ++c) {
      float x[1][8], g[1][8], p[8];
      load_pair<T, AL, TPR, DYF, CK>(dY, X, codes, scales, r, d, t, c, x, g);
      load_param<T, AL, TPR>(w, p_f32, d, t, c, 1.0f, p);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gw = g[0][j] * p[j];  // (past the row's end dy is 0)
        s1 = __builtin_fmaf(gw, (x[0][j] - mu) * rs, s1);
        s2 += gw;
      }
    }
    row_sum2<TPR>(s1, s2, red);
    s1 = quotient(s1, fd, inv_d);
    s2 = mean ? quotient(s2, fd, inv_d) : 0.0f;
    for (int c = 0; c < chunks; ++c) {
      float x[1][8], g[1][8], p[8];
      load_pair<T, AL, TPR, DYF, CK>(dY, X, codes, scales, r, d, t, c, x, g);
      load_param<T, AL, TPR>(w, p_f32, d, t, c, 1.0f, p);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[0][j] = rs * (g[0][j] * p[j] - s2 - (x[0][j] - mu) * rs * s1);
      store_row<T, AL, TPR, 1>(dX + r * d + c * 8 * TPR, d - c * 8 * TPR, t, x);
    }
  }
}

// dw and db of 2048 columns over the rows of slab blockIdx.y
template <typename T, bool AL, bool DYF, bool CK>
__global__ void __launch_bounds__(256)
k_norm_cols(const void* __restrict__ dY, const T* __restrict__ X, const int8_t* __restrict__ codes,
            const uint8_t* __restrict__ scales, const float* __restrict__ mean, const float* __restrict__ rstd,
            int64_t m, int d, float* __restrict__ part_w, float* __restrict__ part_b) {
  constexpr int TPR = 256;
  const int t = (int)threadIdx.x, c = (int)blockIdx.x, base = c * 8 * TPR;
  const int64_t per = (m + gridDim.y - 1) / gridDim.y, r0 = per * blockIdx.y, r1 = r0 + per < m ? r0 + per : m;
  float aw[1][8] = {}, ab[1][8] = {};
#pragma unroll 4
  for (int64_t r = r0; r < r1; ++r) {
    float x[1][8], g[1][8];
    load_pair<T, AL, TPR, DYF, CK>(dY, X, codes, scales, r, d, t, c, x, g);
    const float mu = mean ? mean[r] : 0.0f, rs = rstd[r];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      aw[0][j] = __builtin_fmaf(g[0][j], (x[0][j] - mu) * rs, aw[0][j]);
      ab[0][j] += g[0][j];
    }
  }
  if (part_w) store_row<float, AL, TPR, 1>(part_w + (int64_t)blockIdx.y * d + base, d - base, t, aw);
  if (part_b) store_row<float, AL, TPR, 1>(part_b + (int64_t)blockIdx.y * d + base, d - base, t, ab);
}

// out[j] = (accumulate ? out[j] : 0) + the sum over the blocks' rows of part:
// 64 columns per block, 16 slices of rows summed apart and then in slice order.
// blockIdx.y: dw, db (the one that is wanted when there is one)
__global__ void __launch_bounds__(1024) k_norm_reduce(const float* __restrict__ part, int rows, int d,
                                                      float* __restrict__ out0, float* __restrict__ out1,
                                                      int accumulate) {
  __shared__ float sm[16][64];
  const int lane = (int)(threadIdx.x & 63), sl = (int)(threadIdx.x >> 6);
  const int j = (int)blockIdx.x * 64 + lane;
  part += (int64_t)blockIdx.y * rows * d;
  float* out = blockIdx.y ? out1 : out0;
  float a = 0.0f;
  if (j < d) {
    int r = sl;
    for (; r + 112 < rows; r += 128) {  // eight loads in flight
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = part[(int64_t)(r + 16 * k) * d + j];
#pragma unroll
      for (int k = 0; k < 8; ++k) a += v[k];
    }
    for (; r < rows; r += 16) a += part[(int64_t)r * d + j];
  }
  sm[sl][lane] = a;
  __syncthreads();
  if (sl == 0 && j < d) {
#pragma unroll
    for (int i = 1; i < 16; ++i) a += sm[i][lane];
    out[j] = accumulate ? out[j] + a : a;
  }
}

// (threads per row, chunks per thread) by the row's length: one wave up to
// 2048 columns, then 256 threads up to 8192 and 512 up to 16384, then 1024
struct NormShape {
  int tpr, nch;
};
constexpr int64_t WIDE = 16384;  // beyond: k_norm_bwd_wide, k_norm_cols
NormShape shape_of(int64_t d) {
  if (d <= 512) return {64, 1};
  if (d <= 1024) return {64, 2};
  if (d <= 2048) return {64, 4};
  if (d <= 4096) return {256, 2};
  if (d <= 8192) return {256, 4};
  if (d <= 16384) return {512, 4};
  return {1024, 8};
}

template <typename F>
hipError_t with_shape(int64_t d, F&& f) {
  const NormShape s = shape_of(d);
  if (s.tpr == 64) {
    if (s.nch == 1) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    if (s.nch == 2) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  }
  if (s.tpr == 256) {
    if (s.nch == 2) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
  }
  if (s.tpr == 512) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
}

template <typename T>
hipError_t norm_fwd_t(const NormArgs& a, const T* X, T* Y, float* mean, float* rstd, int8_t* codes, uint8_t* scales,
                      hipStream_t s) {
  return with_shape(a.d, [&](auto tpr, auto nch) {
    constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value;
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const auto kern = a.d % 8 == 0 ? k_norm_fwd<T, true, TPR, NCH> : k_norm_fwd<T, false, TPR, NCH>;
    // a launch has fewer than 2^32 threads: at most 2^21 rows of up to 1024
    constexpr int64_t most = int64_t(1) << 21;
    hipError_t e = hipSuccess;
    for (int64_t r = 0; r < a.m && e == hipSuccess; r += most) {
      const int64_t m = a.m - r < most ? a.m - r : most;
      hipLaunchKernelGGL(kern, dim3((unsigned)((m + RPB - 1) / RPB)), dim3(TPR < 256 ? 256 : TPR), 0, s, X + r * a.d,
                         a.w, a.bias, a.p_f32, m, (int)a.d, a.layer, a.eps, Y + r * a.d, mean ? mean + r : nullptr,
                         rstd + r, codes ? codes + r * a.d : nullptr, scales ? scales + r * (a.d / 32) : nullptr);
      e = hipGetLastError();
    }
    return e;
  });
}

// Blocks of the backward walk, each with one partial row of dw and of db: at
// most two per CU.
int64_t bwd_blocks(int64_t m, int64_t d) {
  if (d > WIDE) return m < 64 ? m : 64;  // slabs of k_norm_cols
  const int rpb = shape_of(d).tpr < 256 ? 256 / shape_of(d).tpr : 1;
  const int64_t need = (m + rpb - 1) / rpb;
  return need < 512 ? need : 512;
}

struct NormBwd {
  const void* dY;
  bool dy_f32;
  const void* X;
  const int8_t* codes;
  const uint8_t* scales;
  const float *mean, *rstd;
  void* dX;
  float *part_w, *part_b;
};

template <typename T, bool AL, bool DYF, bool CK>
hipError_t norm_bwd_wide(const NormArgs& a, const NormBwd& q, hipStream_t s) {
  if (q.dX) {
    hipLaunchKernelGGL((k_norm_bwd_wide<T, AL, DYF, CK>), dim3((unsigned)(a.m < 512 ? a.m : 512)), dim3(1024), 0, s,
                       q.dY, (const T*)q.X, q.codes, q.scales, a.w, a.p_f32, q.mean, q.rstd, a.m, (int)a.d, (T*)q.dX);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!q.part_w && !q.part_b) return hipSuccess;
  const dim3 grid((unsigned)((a.d + 2047) / 2048), (unsigned)bwd_blocks(a.m, a.d));
  hipLaunchKernelGGL((k_norm_cols<T, AL, DYF, CK>), grid, dim3(256), 0, s, q.dY, (const T*)q.X, q.codes, q.scales,
                     q.mean, q.rstd, a.m, (int)a.d, q.part_w, q.part_b);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_bwd_t(const NormArgs& a, const NormBwd& q, hipStream_t s) {
  constexpr bool F = __is_same(T, float);  // (an fp32 dY of fp32 rows is of their own type)
  const bool f = q.dy_f32 && !F;
  if (a.d > WIDE) {
    if (q.codes) return f ? norm_bwd_wide<T, true, !F, true>(a, q, s) : norm_bwd_wide<T, true, false, true>(a, q, s);
    if (a.d % 8 == 0)
      return f ? norm_bwd_wide<T, true, !F, false>(a, q, s) : norm_bwd_wide<T, true, false, false>(a, q, s);
    return f ? norm_bwd_wide<T, false, !F, false>(a, q, s) : norm_bwd_wide<T, false, false, false>(a, q, s);
  }
  return with_shape(a.d, [&](auto tpr, auto nch) {
    constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value;
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, dim3((unsigned)bwd_blocks(a.m, a.d)), dim3(TPR < 256 ? 256 : TPR), 0, s, q.dY,
                         (const T*)q.X, q.codes, q.scales, a.w, a.p_f32, q.mean, q.rstd, a.m, (int)a.d, (T*)q.dX,
                         q.part_w, q.part_b);
      return hipGetLastError();
    };
    if constexpr (TPR == 1024) {
      return hipErrorNotSupported;  // (no such call comes here)
    } else {
      if (q.codes)
        return f ? go(k_norm_bwd<T, true, TPR, NCH, !F, true>) : go(k_norm_bwd<T, true, TPR, NCH, false, true>);
      if (a.d % 8 == 0)
        return f ? go(k_norm_bwd<T, true, TPR, NCH, !F, false>) : go(k_norm_bwd<T, true, TPR, NCH, false, false>);
      return f ? go(k_norm_bwd<T, false, TPR, NCH, !F, false>) : go(k_norm_bwd<T, false, TPR, NCH, false, false>);
    }
  });
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, const void* X, int x_dtype, void* Y, float* mean, float* rstd,
                           int8_t* codes, uint8_t* scales, hipStream_t s) {
  if (x_dtype == DT_F32) return norm_fwd_t(a, (const float*)X, (float*)Y, mean, rstd, codes, scales, s);
  if (x_dtype == DT_F16) return norm_fwd_t(a, (const half_t*)X, (half_t*)Y, mean, rstd, codes, scales, s);
  return norm_fwd_t(a, (const bf16_t*)X, (bf16_t*)Y, mean, rstd, codes, scales, s);
}

size_t norm_bwd_part_bytes(int64_t m, int64_t d) { return (size_t)bwd_blocks(m, d) * (size_t)d * 4; }

hipError_t launch_norm_bwd(const NormArgs& a, const void* dY, int dy_dtype, const void* X, int x_dtype,
                           const int8_t* codes, const uint8_t* scales, const float* mean, const float* rstd, void* dX,
                           float* dw, float* db, int accumulate, float* part, hipStream_t s) {
  const int64_t rows = bwd_blocks(a.m, a.d);
  const NormBwd q{dY,   dy_dtype == DT_F32,    X,
                  codes, scales,                mean,
                  rstd, dX,                    dw ? part : nullptr,
                  db ? part + (dw ? rows * a.d : 0) : nullptr};
  hipError_t e;
  if (x_dtype == DT_F32) e = norm_bwd_t<float>(a, q, s);
  else if (x_dtype == DT_F16) e = norm_bwd_t<half_t>(a, q, s);
  else e = norm_bwd_t<bf16_t>(a, q, s);
  if (e != hipSuccess || (!dw && !db)) return e;
  hipLaunchKernelGGL(k_norm_reduce, dim3((unsigned)((a.d + 63) / 64), dw && db ? 2 : 1), dim3(1024), 0, s, part,
                     (int)rows, (int)a.d, dw ? dw : db, db, accumulate);
  return hipGetLastError();
}

}  // namespace skm
