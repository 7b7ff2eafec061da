// Matrix-core backward of the sketched matmul: the plain matmul's instances of
// the kernels in skm_gemm_bwd.h.
#include "skm_gemm_bwd.h"

namespace skm {

namespace {

template <typename TX, typename TL>
hipError_t dx_t(const TX* dY, const uint8_t* idx, const TL* lut, const Problem& p, float* dX, const int32_t* rexp,
                hipStream_t s) {
  switch (p.b) {
    case 2: return dx_b<2>(dY, idx, lut, p, dX, rexp, Whole{}, s);
    case 3: return dx_b<3>(dY, idx, lut, p, dX, rexp, Whole{}, s);
    default: return dx_b<4>(dY, idx, lut, p, dX, rexp, Whole{}, s);
  }
}

template <int B, typename TX>
hipError_t dlut_b(const TX* dY, const TX* X, const uint8_t* idx, const Problem& p, float* dLUT, int accumulate,
                  float* part, hipStream_t s) {
  // DMA staging: whole 32-token steps and 16-byte aligned dY rows
  if (p.m % DL_BK == 0 && p.n % 8 == 0)
    return dlut_dma_launch<B, TX>(dY, X, idx, p, dLUT, accumulate, part, s);
  if (p.n % 8 == 0) return dlut_launch<B, TX, true>(dY, X, idx, p, dLUT, accumulate, part, s);
  return dlut_launch<B, TX, false>(dY, X, idx, p, dLUT, accumulate, part, s);
}

template <typename TX>
hipError_t dlut_t(const TX* dY, const TX* X, const uint8_t* idx, const Problem& p, float* dLUT, int accumulate,
                  float* part, hipStream_t s) {
  switch (p.b) {
    case 2: return dlut_b<2>(dY, X, idx, p, dLUT, accumulate, part, s);
    case 3: return dlut_b<3>(dY, X, idx, p, dLUT, accumulate, part, s);
    default: return dlut_b<4>(dY, X, idx, p, dLUT, accumulate, part, s);
  }
}

}  // namespace

bool gemm_bwd_supported(const Problem& p) { return p.d <= (int64_t(1) << 20); }

size_t dlut_partial_bytes(const Problem& p) {
  const DlutSplit sp = dlut_split_of(p);
  return sp.parts() > 1 ? (size_t)sp.parts() * (size_t)(p.n * p.gpr * p.k()) * 4 : 0;
}

hipError_t launch_gemm_dx(const void* dY, int io_dtype, const uint8_t* idx, const void* lut, int lut_dtype,
                          const Problem& p, float* dX, const int32_t* rexp, hipStream_t s) {
  if (io_dtype == DT_F16 && lut_dtype == DT_F16)
    return dx_t((const half_t*)dY, idx, (const half_t*)lut, p, dX, nullptr, s);
  if (io_dtype == DT_BF16 && lut_dtype == DT_F16)
    return dx_t((const bf16_t*)dY, idx, (const half_t*)lut, p, dX, rexp, s);
  if (io_dtype == DT_F16 && lut_dtype == DT_BF16)
    return dx_t((const half_t*)dY, idx, (const bf16_t*)lut, p, dX, nullptr, s);
  return dx_t((const bf16_t*)dY, idx, (const bf16_t*)lut, p, dX, nullptr, s);
}

hipError_t launch_gemm_dlut(const void* dY, const void* X, int io_dtype, const uint8_t* idx, const Problem& p,
                            float* dLUT, int accumulate, float* part, hipStream_t s) {
  if (io_dtype == DT_F16) return dlut_t((const half_t*)dY, (const half_t*)X, idx, p, dLUT, accumulate, part, s);
  return dlut_t((const bf16_t*)dY, (const bf16_t*)X, idx, p, dLUT, accumulate, part, s);
}

}  // namespace skm
