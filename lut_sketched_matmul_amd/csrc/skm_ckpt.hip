// 8-bit activation checkpoints: writing (k_act_quant) and reading back
// (k_act_dequant). The format is in skm_quant.h.
//
// Rows are whole blocks of 32 columns, so a matrix is one flat run of blocks
// and each kernel a stream: a lane takes 8 columns (four lanes per block, whose
// largest magnitude two quad permutes find), kept in registers between the
// maximum and the rounding, so every value is read once.
#include "skm_launch.h"
#include "skm_quant.h"

namespace skm {

namespace {

template <typename T>
__global__ void __launch_bounds__(256) k_act_quant(const T* __restrict__ X, int64_t chunks, int8_t* __restrict__ codes,
                                                   uint8_t* __restrict__ scales) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;  // chunks is a multiple of 4: quads stay whole
  float v[8];
  load8<T>(X + c * 8, v);
  const uint32_t s = ckpt_exp_of<T>(quad_max(top8(v)));
  *reinterpret_cast<u32x2*>(codes + c * 8) = ckpt_pack8(v, s);
  if ((threadIdx.x & 3) == 0) scales[c >> 2] = (uint8_t)s;
}

template <typename T>
__global__ void __launch_bounds__(256) k_act_dequant(const int8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales, int64_t chunks,
                                                     T* __restrict__ X) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;
  float v[8];
  ckpt_unpack8(*reinterpret_cast<const u32x2*>(codes + c * 8), scales[c >> 2], v);
  store8<T>(X + c * 8, v);
}

}  // namespace

hipError_t launch_act_quant(const void* X, int x_dtype, int64_t count, int8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t chunks = count / 8;
  const dim3 grid((unsigned)((chunks + 255) / 256));
  if (x_dtype == DT_F32)
    hipLaunchKernelGGL(k_act_quant<float>, grid, dim3(256), 0, s, (const float*)X, chunks, codes, scales);
  else if (x_dtype == DT_F16)
    hipLaunchKernelGGL(k_act_quant<half_t>, grid, dim3(256), 0, s, (const half_t*)X, chunks, codes, scales);
  else
    hipLaunchKernelGGL(k_act_quant<bf16_t>, grid, dim3(256), 0, s, (const bf16_t*)X, chunks, codes, scales);
  return hipGetLastError();
}

hipError_t launch_act_dequant(const int8_t* codes, const uint8_t* scales, int64_t count, void* X, int x_dtype,
                              hipStream_t s) {
  const int64_t chunks = count / 8;
  const dim3 grid((unsigned)((chunks + 255) / 256));
  if (x_dtype == DT_F32)
    hipLaunchKernelGGL(k_act_dequant<float>, grid, dim3(256), 0, s, codes, scales, chunks, (float*)X);
  else if (x_dtype == DT_F16)
    hipLaunchKernelGGL(k_act_dequant<half_t>, grid, dim3(256), 0, s, codes, scales, chunks, (half_t*)X);
  else
    hipLaunchKernelGGL(k_act_dequant<bf16_t>, grid, dim3(256), 0, s, codes, scales, chunks, (bf16_t*)X);
  return hipGetLastError();
}

}  // namespace skm
