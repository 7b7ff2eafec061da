// The backward products with the caller's own operand layout (DxPiece of
// skm_gemm_bwd.h, DlPiece of skm_gemm_dlut.h): ranges of the weight rows,
// padded token rows, a token count on the device.
#include "skm_gemm_dlut.h"

namespace skm {

namespace {

template <typename TX, typename TL>
hipError_t dx_piece_t(const void* dY, const uint8_t* idx, const void* lut, const Problem& p, float* dX,
                      const int32_t* rexp, const DxPiece& pa, hipStream_t s) {
  const TX* y = (const TX*)dY;
  const TL* l = (const TL*)lut;
  if (p.b == 2) return dx_b<2, TX, TL>(y, idx, l, p, dX, rexp, pa, s);
  if (p.b == 3) return dx_b<3, TX, TL>(y, idx, l, p, dX, rexp, pa, s);
  return dx_b<4, TX, TL>(y, idx, l, p, dX, rexp, pa, s);
}

template <typename TX, bool TWO>
hipError_t dlut_piece_t(const void* hi, const void* lo, const void* X, const uint8_t* idx, const Problem& p,
                        float* dLUT, int accumulate, float* part, const DlutPiece& q, hipStream_t s) {
  const TX* y = (const TX*)hi;
  const TX* x = (const TX*)X;
  const DlPiece pa{q.count, q.ld, TWO ? (const TX*)lo - y : 0, q.inv_scale, q.zeros};
  if (p.b == 2) return dlut_piece_launch<2, TX, TWO>(y, x, idx, p, dLUT, accumulate, part, pa, s);
  if (p.b == 3) return dlut_piece_launch<3, TX, TWO>(y, x, idx, p, dLUT, accumulate, part, pa, s);
  return dlut_piece_launch<4, TX, TWO>(y, x, idx, p, dLUT, accumulate, part, pa, s);
}

}  // namespace

// Ranges of the weight rows so that dX's (256-token, 256-column) tiles fill the
// 256 CUs: the count that minimises rounds of 256 blocks times 64-row steps per
// block, at least 4 steps each and at most two rounds (the ranges' sums are
// written and read once more, 4 bytes per output and range).
DxRanges dx_ranges(const Problem& p) {
  const int64_t steps = (p.n + 63) / 64;
  const int64_t nb0 = (p.m + 255) / 256 * ((p.d + 255) / 256);
  int64_t best = 1, cost = (nb0 + 255) / 256 * steps;
  for (int64_t c = 2; c * 4 <= steps && nb0 * c <= 512; ++c) {
    const int64_t k = (nb0 * c + 255) / 256 * ((steps + c - 1) / c);
    if (k < cost) {
      cost = k;
      best = c;
    }
  }
  const int64_t rows = (steps + best - 1) / best * 64;
  return {(int)((p.n + rows - 1) / rows), rows};
}

hipError_t launch_dx_piece(const void* dY, int io_dtype, const uint8_t* idx, const void* lut, int lut_dtype,
                           const Problem& p, float* dX, const int32_t* rexp, const int32_t* count, int64_t ld,
                           int accumulate, const DxRanges& r, const DxPlan* plan, int64_t blocks, hipStream_t s) {
  if (accumulate && scaled_pair(io_dtype == DT_BF16, lut_dtype == DT_F16)) return hipErrorNotSupported;
  if (!plan) blocks = (p.m + DX_BM - 1) / DX_BM * ((p.d + DX_BN - 1) / DX_BN) * r.count;
  const DxPiece pa{count, ld, accumulate, r.count, r.rows, p.m * p.d, plan, (unsigned)blocks};
  if (io_dtype == DT_F16 && lut_dtype == DT_F16)
    return dx_piece_t<half_t, half_t>(dY, idx, lut, p, dX, nullptr, pa, s);
  if (io_dtype == DT_BF16 && lut_dtype == DT_F16)
    return dx_piece_t<bf16_t, half_t>(dY, idx, lut, p, dX, rexp, pa, s);
  if (io_dtype == DT_F16) return dx_piece_t<half_t, bf16_t>(dY, idx, lut, p, dX, nullptr, pa, s);
  return dx_piece_t<bf16_t, bf16_t>(dY, idx, lut, p, dX, nullptr, pa, s);
}

hipError_t launch_dlut_piece(const void* hi, const void* lo, const void* X, int io_dtype, const uint8_t* idx,
                             const Problem& p, float* dLUT, int accumulate, float* part, const DlutPiece& q,
                             hipStream_t s) {
  // (two addends are f16 and their rows past the tokens zeros)
  if (lo && (io_dtype != DT_F16 || q.zeros)) return hipErrorNotSupported;
  if (lo) return dlut_piece_t<half_t, true>(hi, lo, X, idx, p, dLUT, accumulate, part, q, s);
  if (io_dtype == DT_F16) return dlut_piece_t<half_t, false>(hi, lo, X, idx, p, dLUT, accumulate, part, q, s);
  return dlut_piece_t<bf16_t, false>(hi, lo, X, idx, p, dLUT, accumulate, part, q, s);
}

}  // namespace skm
