// Dropout of a tensor, with the residual it is added to:
//   y_i = [residual_i +] (keep_i ? x_i / (1 - p) : 0)
// keep_i from a counter (skm_philox.h): the backward pass is the same call on
// the output's gradient, and no mask is stored. p is the multiple of 2^-16
// nearest to the caller's, so the share that stays is exactly 1 - p.
//
// Values that do not stay are selected away, not multiplied by zero (they may
// be infinities or NaN). fp32 values are divided by 1 - p (a product with
// the rounded quotient would be off by a further half step); 16-bit ones are
// multiplied by it, 2^-24 before their own rounding to 2^-9 or 2^-12.
//
// One thread takes the eight values of one generator call, 16 bytes of a
// 16-bit tensor. Bound by memory: 8192 x 4096 bf16 24 us (5.6 TB/s; the generator's
// ten rounds hide behind the loads), with a residual 38 us (5.3), both what a large copy
// reaches; one launch of 2.7 us for a few rows.
#include "skm_launch.h"
#include "skm_philox.h"
#include "skm_quant.h"

namespace skm {

namespace {

constexpr int THREADS = 256;
constexpr int64_t MAX_BLOCKS = int64_t(1) << 20;

template <typename T>
__device__ __forceinline__ float dropped(float x, bool stays, float stay, float inv) {
  if constexpr (__is_same(T, float)) return stays ? x / stay : 0.f;
  return stays ? x * inv : 0.f;
}

template <typename T, bool RES>
__global__ __launch_bounds__(THREADS) void k_dropout(const T* __restrict__ X, const T* __restrict__ R,
                                                     int64_t count, uint32_t threshold, float stay, float inv,
                                                     const int64_t* __restrict__ seed, T* __restrict__ Y) {
  const Philox g = threshold ? philox_of(seed) : Philox{0u, 0u, 0u, 0u};
  const int64_t step = (int64_t)gridDim.x * THREADS;
  for (int64_t b = (int64_t)blockIdx.x * THREADS + threadIdx.x; b * 8 < count; b += step) {
    const int64_t i = b * 8;
    const bool whole = i + 8 <= count;
    float x[8], r[8];
    if (whole) {
      load8<T>(X + i, x);
      if (RES) load8<T>(R + i, r);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = i + j < count ? to_f32(X[i + j]) : 0.f;
        r[j] = RES && i + j < count ? to_f32(R[i + j]) : 0.f;
      }
    }
    const u32x4 u = threshold ? philox_block(g, (uint64_t)b) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = dropped<T>(x[j], philox_stays(u, j, threshold), stay, inv);
      x[j] = RES ? r[j] + y : y;
    }
    if (whole) {
      store8<T>(Y + i, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < count) Y[i + j] = from_f32<T>(x[j]);
    }
  }
}

template <typename T>
hipError_t dropout_t(const void* X, const void* R, int64_t count, const Dropout& d, void* Y, hipStream_t s) {
  const int64_t blocks = (count + 8 * THREADS - 1) / (8 * THREADS);
  const dim3 grid((unsigned)(blocks < MAX_BLOCKS ? blocks : MAX_BLOCKS)), block(THREADS);
  if (R)
    hipLaunchKernelGGL((k_dropout<T, true>), grid, block, 0, s, (const T*)X, (const T*)R, count, d.threshold,
                       d.stay(), d.inv(), d.seed, (T*)Y);
  else
    hipLaunchKernelGGL((k_dropout<T, false>), grid, block, 0, s, (const T*)X, (const T*)nullptr, count, d.threshold,
                       d.stay(), d.inv(), d.seed, (T*)Y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* X, int x_dtype, const void* residual, int64_t count, const Dropout& d, void* Y,
                          hipStream_t s) {
  if (x_dtype == DT_F32) return dropout_t<float>(X, residual, count, d, Y, s);
  if (x_dtype == DT_F16) return dropout_t<half_t>(X, residual, count, d, Y, s);
  return dropout_t<bf16_t>(X, residual, count, d, Y, s);
}

}  // namespace skm
