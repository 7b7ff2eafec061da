// Layer norm and root-mean-square norm of the rows of X [m][d], forward and
// backward (the norm in front of a sketched layer).
//
//   layer: mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r
//   rms:   mu = 0,       r = 1 / sqrt(mean(x^2) + eps),        xh = x r
//   y  = xh w + b
//   dx = r (g - xh mean(g xh) - [layer] mean(g)),  g = dy w
//   dw = sum_rows dy xh,   db = sum_rows dy
//
// All arithmetic is fp32. A row is read once and stays in registers: TPR
// threads of E = 8 NCH elements each, so the variance is taken from the
// centred values (no cancellation) without a second read. Rows of whole
// 8-column chunks (AL) move 8 consecutive columns per lane; other widths take
// the same kernels with column j TPR + t in element j of thread t.
//
// Backward: each block walks rows blockIdx, blockIdx + grid, ... and keeps its
// columns' dw and db sums in registers; the block's sums go to the workspace
// and k_norm_reduce adds them per column in block order (deterministic, no
// atomics).
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

// a weight or bias row (fp32 or T; NULL gives `fill`)
template <typename T, bool AL, int TPR, int NCH>
__device__ __forceinline__ void load_param(const void* p, int p_f32, int d, int t, float fill, float (&v)[NCH][8]) {
  if (!p) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = fill;
  } else if (p_f32) {
    load_row<float, AL, TPR, NCH>((const float*)p, d, t, v);
  } else {
    load_row<T, AL, TPR, NCH>((const T*)p, d, t, v);
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
  const float inv_d = 1.0f / (float)d;
  float mu = 0.0f, z = 0.0f;
  if (layer) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) mu += x[c][j];
    row_sum2<TPR>(mu, z, red);
    mu *= inv_d;
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
  const float rs = 1.0f / sqrtf(var * inv_d + eps);
  if (t == 0) {
    rstd[r] = rs;
    if (mean) mean[r] = mu;
  }
  float p[NCH][8];
  load_param<T, AL, TPR, NCH>(w, p_f32, d, t, 1.0f, p);
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) x[c][j] = x[c][j] * rs * p[c][j];
  if (bias) {
    load_param<T, AL, TPR, NCH>(bias, p_f32, d, t, 0.0f, p);
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[c][j] += p[c][j];
  }
  store_row<T, AL, TPR, NCH>(Y + r * d, d, t, x);
  if constexpr (AL) {
    if (codes) {  // d is a multiple of 32: the four lanes of a block are in range together
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int j0 = col_of<AL, TPR>(t, c, 0);
        if (j0 >= d) continue;
        // the checkpoint is of Y as stored
#pragma unroll
        for (int j = 0; j < 8; ++j) x[c][j] = to_f32(from_f32<T>(x[c][j]));
        const uint32_t s = ckpt_exp_of<T>(quad_max(top8(x[c])));
        *reinterpret_cast<u32x2*>(codes + r * d + j0) = ckpt_pack8(x[c], s);
        if ((t & 3) == 0) scales[(r * d + j0) >> 5] = (uint8_t)s;
      }
    }
  }
}

template <typename T, bool AL, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
k_norm_bwd(const void* __restrict__ dY, int dy_f32, const T* __restrict__ X, const int8_t* __restrict__ codes,
           const uint8_t* __restrict__ scales, const void* __restrict__ w, int p_f32, const float* __restrict__ mean,
           const float* __restrict__ rstd, int64_t m, int d, T* __restrict__ dX, float* __restrict__ part_w,
           float* __restrict__ part_b) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[2 * (TPR / 64)];
  const int t = (int)(threadIdx.x % TPR);
  const float inv_d = 1.0f / (float)d;
  float p[NCH][8], aw[NCH][8], ab[NCH][8];
  load_param<T, AL, TPR, NCH>(w, p_f32, d, t, 1.0f, p);
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[c][j] = ab[c][j] = 0.0f;
  for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; r < m; r += (int64_t)gridDim.x * RPB) {
    float x[NCH][8], g[NCH][8];
    if (dy_f32) load_row<float, AL, TPR, NCH>((const float*)dY + r * d, d, t, g);
    else load_row<T, AL, TPR, NCH>((const T*)dY + r * d, d, t, g);
    if (AL && codes) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int j0 = col_of<AL, TPR>(t, c, 0);
        if (j0 < d) {
          ckpt_unpack8(*reinterpret_cast<const u32x2*>(codes + r * d + j0), scales[(r * d + j0) >> 5], x[c]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[c][j] = 0.0f;
        }
      }
    } else {
      load_row<T, AL, TPR, NCH>(X + r * d, d, t, x);
    }
    const float mu = mean ? mean[r] : 0.0f, rs = rstd[r];
    float s1 = 0.0f, s2 = 0.0f;  // sums of g xh and of g, g = dy w
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (x[c][j] - mu) * rs;  // (past the row's end dy is 0)
        aw[c][j] = __builtin_fmaf(g[c][j], xh, aw[c][j]);
        ab[c][j] += g[c][j];
        g[c][j] *= p[c][j];
        x[c][j] = xh;
        s1 = __builtin_fmaf(g[c][j], xh, s1);
        s2 += g[c][j];
      }
    if (dX) {
      row_sum2<TPR>(s1, s2, red);
      s1 *= inv_d;
      s2 = mean ? s2 * inv_d : 0.0f;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[c][j] = rs * (g[c][j] - s2 - x[c][j] * s1);
      store_row<T, AL, TPR, NCH>(dX + r * d, d, t, x);
    }
  }
  // the block's sums, one partial row per row slot of the block
  const int64_t slot = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (part_w) store_row<float, AL, TPR, NCH>(part_w + slot * d, d, t, aw);
  if (part_b) store_row<float, AL, TPR, NCH>(part_b + slot * d, d, t, ab);
}

// out[j] = (accumulate ? out[j] : 0) + sum over the partial rows, in order:
// 64 columns per block, 16 slices of rows summed apart and then in slice order
__global__ void __launch_bounds__(1024) k_norm_reduce(const float* __restrict__ part, int rows, int d,
                                                      float* __restrict__ out, int accumulate) {
  __shared__ float sm[16][64];
  const int lane = (int)(threadIdx.x & 63), sl = (int)(threadIdx.x >> 6);
  const int j = (int)blockIdx.x * 64 + lane;
  float a = 0.0f;
  if (j < d)
    for (int r = sl; r < rows; r += 16) a += part[(int64_t)r * d + j];
  sm[sl][lane] = a;
  __syncthreads();
  if (sl == 0 && j < d) {
#pragma unroll
    for (int i = 1; i < 16; ++i) a += sm[i][lane];
    out[j] = accumulate ? out[j] + a : a;
  }
}

// (threads per row, chunks per thread) by the row's length: one wave up to
// 2048 columns, then 256 threads up to 16384, then 1024
struct NormShape {
  int tpr, nch;
};
NormShape shape_of(int64_t d) {
  if (d <= 512) return {64, 1};
  if (d <= 2048) return {64, 4};
  if (d <= 4096) return {256, 2};
  if (d <= 8192) return {256, 4};
  if (d <= 16384) return {256, 8};
  return {1024, 8};
}

template <typename F>
hipError_t with_shape(int64_t d, F&& f) {
  const NormShape s = shape_of(d);
  if (s.tpr == 64) return s.nch == 1 ? f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{})
                                     : f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  if (s.tpr == 256) {
    if (s.nch == 2) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    if (s.nch == 4) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 8>{});
  }
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
}

template <typename T>
hipError_t norm_fwd_t(const NormArgs& a, const T* X, T* Y, float* mean, float* rstd, int8_t* codes, uint8_t* scales,
                      hipStream_t s) {
  return with_shape(a.d, [&](auto tpr, auto nch) {
    constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value;
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)((a.m + RPB - 1) / RPB)), block(TPR < 256 ? 256 : TPR);
    if (a.d % 8 == 0)
      hipLaunchKernelGGL((k_norm_fwd<T, true, TPR, NCH>), grid, block, 0, s, X, a.w, a.bias, a.p_f32, a.m, (int)a.d,
                         a.layer, a.eps, Y, mean, rstd, codes, scales);
    else
      hipLaunchKernelGGL((k_norm_fwd<T, false, TPR, NCH>), grid, block, 0, s, X, a.w, a.bias, a.p_f32, a.m, (int)a.d,
                         a.layer, a.eps, Y, mean, rstd, codes, scales);
    return hipGetLastError();
  });
}

// blocks of the backward walk
int64_t bwd_blocks(int64_t m, int64_t d) {
  const int rpb = shape_of(d).tpr < 256 ? 256 / shape_of(d).tpr : 1;
  const int64_t need = (m + rpb - 1) / rpb;
  return need < 512 ? need : 512;
}
int64_t bwd_slots(int64_t m, int64_t d) {
  const int rpb = shape_of(d).tpr < 256 ? 256 / shape_of(d).tpr : 1;
  return bwd_blocks(m, d) * rpb;
}

template <typename T>
hipError_t norm_bwd_t(const NormArgs& a, const void* dY, int dy_f32, const T* X, const int8_t* codes,
                      const uint8_t* scales, const float* mean, const float* rstd, T* dX, float* part_w, float* part_b,
                      hipStream_t s) {
  return with_shape(a.d, [&](auto tpr, auto nch) {
    constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value;
    const dim3 grid((unsigned)bwd_blocks(a.m, a.d)), block(TPR < 256 ? 256 : TPR);
    if (a.d % 8 == 0)
      hipLaunchKernelGGL((k_norm_bwd<T, true, TPR, NCH>), grid, block, 0, s, dY, dy_f32, X, codes, scales, a.w,
                         a.p_f32, mean, rstd, a.m, (int)a.d, dX, part_w, part_b);
    else
      hipLaunchKernelGGL((k_norm_bwd<T, false, TPR, NCH>), grid, block, 0, s, dY, dy_f32, X, codes, scales, a.w,
                         a.p_f32, mean, rstd, a.m, (int)a.d, dX, part_w, part_b);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, const void* X, int x_dtype, void* Y, float* mean, float* rstd,
                           int8_t* codes, uint8_t* scales, hipStream_t s) {
  if (x_dtype == DT_F32) return norm_fwd_t(a, (const float*)X, (float*)Y, mean, rstd, codes, scales, s);
  if (x_dtype == DT_F16) return norm_fwd_t(a, (const half_t*)X, (half_t*)Y, mean, rstd, codes, scales, s);
  return norm_fwd_t(a, (const bf16_t*)X, (bf16_t*)Y, mean, rstd, codes, scales, s);
}

size_t norm_bwd_part_bytes(int64_t m, int64_t d) { return (size_t)bwd_slots(m, d) * (size_t)d * 4; }

hipError_t launch_norm_bwd(const NormArgs& a, const void* dY, int dy_dtype, const void* X, int x_dtype,
                           const int8_t* codes, const uint8_t* scales, const float* mean, const float* rstd, void* dX,
                           float* dw, float* db, int accumulate, float* part, hipStream_t s) {
  const int64_t slots = bwd_slots(a.m, a.d);
  float* pw = dw ? part : nullptr;
  float* pb = db ? part + (dw ? slots * a.d : 0) : nullptr;
  const int f32 = dy_dtype == DT_F32;
  hipError_t e;
  if (x_dtype == DT_F32)
    e = norm_bwd_t(a, dY, f32, (const float*)X, codes, scales, mean, rstd, (float*)dX, pw, pb, s);
  else if (x_dtype == DT_F16)
    e = norm_bwd_t(a, dY, f32, (const half_t*)X, codes, scales, mean, rstd, (half_t*)dX, pw, pb, s);
  else
    e = norm_bwd_t(a, dY, f32, (const bf16_t*)X, codes, scales, mean, rstd, (bf16_t*)dX, pw, pb, s);
  const dim3 grid((unsigned)((a.d + 63) / 64));
  if (e == hipSuccess && dw) {
    hipLaunchKernelGGL(k_norm_reduce, grid, dim3(1024), 0, s, pw, (int)slots, (int)a.d, dw, accumulate);
    e = hipGetLastError();
  }
  if (e == hipSuccess && db) {
    hipLaunchKernelGGL(k_norm_reduce, grid, dim3(1024), 0, s, pb, (int)slots, (int)a.d, db, accumulate);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace skm
