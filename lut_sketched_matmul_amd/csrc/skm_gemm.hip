// Matrix-core forward pass Y = X W^T for m > 16 tokens: the plain matmul's
// instances of the kernels in skm_gemm_fwd.h.
#include "skm_gemm_fwd.h"

namespace skm {

namespace {

template <typename TX, typename TL>
hipError_t gemm_fwd_t(const TX* X, const uint8_t* idx, const TL* lut, const Problem& p, TX* Y, const int32_t* rexp,
                      hipStream_t s) {
  switch (p.b) {
    case 2: return gemm_fwd_b<2, TX, TL, EpStore<TX>>(X, idx, lut, p, {Y}, rexp, s);
    case 3: return gemm_fwd_b<3, TX, TL, EpStore<TX>>(X, idx, lut, p, {Y}, rexp, s);
    default: return gemm_fwd_b<4, TX, TL, EpStore<TX>>(X, idx, lut, p, {Y}, rexp, s);
  }
}

}  // namespace

bool gemm_fwd_supported(const Problem& p) {
  // group index by multiply-high is exact while units * units-per-group < 2^32
  return p.d <= (int64_t(1) << 20) && p.n * p.m < (int64_t(1) << 62);
}

hipError_t launch_gemm_fwd(const void* X, int x_dtype, const uint8_t* idx, const void* lut, int lut_dtype,
                           const Problem& p, void* Y, const int32_t* rexp, hipStream_t s) {
  if (x_dtype == DT_F16 && lut_dtype == DT_F16)
    return gemm_fwd_t((const half_t*)X, idx, (const half_t*)lut, p, (half_t*)Y, nullptr, s);
  if (x_dtype == DT_BF16 && lut_dtype == DT_F16)
    return gemm_fwd_t((const bf16_t*)X, idx, (const half_t*)lut, p, (bf16_t*)Y, rexp, s);
  if (x_dtype == DT_F16 && lut_dtype == DT_BF16)
    return gemm_fwd_t((const half_t*)X, idx, (const bf16_t*)lut, p, (half_t*)Y, nullptr, s);
  return gemm_fwd_t((const bf16_t*)X, idx, (const bf16_t*)lut, p, (bf16_t*)Y, nullptr, s);
}

}  // namespace skm
