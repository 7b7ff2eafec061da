// Cross entropy backward: dX and dLUT of a piece of the vocabulary, the
// instances of the backward tiles (skm_gemm_bwd.h) on DxPiece / DlPiece.
#include "skm_gemm_bwd.h"
#include "skm_xent.h"

namespace skm {

namespace {

template <typename TL>
hipError_t dx_piece_t(const void* dY, const uint8_t* idx, const void* lut, const Problem& p, float* dX,
                      const DxPiece& pa, hipStream_t s) {
  const TL* y = (const TL*)dY;
  const TL* l = (const TL*)lut;
  if (p.b == 2) return dx_b<2, TL, TL>(y, idx, l, p, dX, nullptr, pa, s);
  if (p.b == 3) return dx_b<3, TL, TL>(y, idx, l, p, dX, nullptr, pa, s);
  return dx_b<4, TL, TL>(y, idx, l, p, dX, nullptr, pa, s);
}

template <typename TX>
hipError_t dlut_piece_t(const void* hi, const void* lo, const void* Xc, const uint8_t* idx, const Problem& p,
                        float* dLUT, int accumulate, float* part, const XentPiece& q, hipStream_t s) {
  const TX* y = (const TX*)hi;
  const TX* x = (const TX*)Xc;
  const DlPiece pa{&q.head->count, q.ld, lo ? (const TX*)lo - y : 0, &q.head->inv_scale};
  if (p.b == 2) return dlut_dma_launch<2, TX>(y, x, idx, p, dLUT, accumulate, part, pa, s);
  if (p.b == 3) return dlut_dma_launch<3, TX>(y, x, idx, p, dLUT, accumulate, part, pa, s);
  return dlut_dma_launch<4, TX>(y, x, idx, p, dLUT, accumulate, part, pa, s);
}

}  // namespace

hipError_t xent_dx(const void* dY, const uint8_t* idx, const void* lut, int lut_dtype, const Problem& p, float* dX,
                   const XentPiece& q, int accumulate, int splits, int64_t split_rows, hipStream_t s) {
  const DxPiece pa{&q.head->count, q.ld, accumulate, splits, split_rows, p.m * p.d};
  if (lut_dtype == DT_F16) return dx_piece_t<half_t>(dY, idx, lut, p, dX, pa, s);
  return dx_piece_t<bf16_t>(dY, idx, lut, p, dX, pa, s);
}

hipError_t xent_dlut(const void* hi, const void* lo, const void* Xc, int x_dtype, const uint8_t* idx,
                     const Problem& p, float* dLUT, int accumulate, float* part, const XentPiece& q, hipStream_t s) {
  if (x_dtype == DT_F16) return dlut_piece_t<half_t>(hi, lo, Xc, idx, p, dLUT, accumulate, part, q, s);
  return dlut_piece_t<bf16_t>(hi, lo, Xc, idx, p, dLUT, accumulate, part, q, s);
}

}  // namespace skm
