// Softmax cross entropy of a sketched vocabulary projection Z = X W^T (W the
// sketched [V][d] head) whose logits Z are never stored.
//
//   lse_t  = log sum_v exp(z_tv)         loss_t = lse_t - z_t,target(t)
//   dz_tv  = dloss_t (exp(z_tv - lse_t) - [v == target(t)])
//   dX = dZ W,   dLUT = sums of dZ^T X over the columns sharing an entry
//
// Forward: the matmul's tiles (skm_gemm_fwd.h) with EpStats, which reduces a
// block's 256 x 256 logits in registers to one (max, sum of exp) pair per
// token; a merge adds the pairs of all vocabulary blocks. The operands of the
// MFMA are exchanged, so that the 64 logits a lane pair holds of a token sit in
// registers and the softmax needs one cross-lane step instead of a reduction
// over 32 lanes per token.
//
// Backward: the logits are computed again a piece of the vocabulary at a time
// and EpGrad turns them into dZ (they would cost as many bytes to keep as to
// recompute flops: at 4096 tokens and 32000 words, 0.5 GB against 0.5 ms). dX
// and dLUT then run on the piece (skm_gemm_bwd.h).
//
// Rounding. dZ is an MFMA operand, so it is 16 bits wide. dX, itself rounded
// to 16 bits, takes dZ rounded once, in the tables' dtype (half a step per
// term). The target's term, which carries most of a token's gradient, keeps its
// remainder in fp32 and k_xent_dx_out adds it times the target's weights. What
// is left is the half step of the other terms, of a token at most about the half
// step that rounds its dX anyway: 2048 bf16 tokens, 128256 words, off by 1.687e-3
// of dX's norm in 64 bits, 1.660e-3 with dZ in fp32 (bf16's rounding of dX alone;
// the median token 1.6e-5 before it); a second addend would double dX's matrix
// work, half of that call. 4096 f16 tokens: 2.11e-4 and 2.07e-4. dLUT
// is fp32: it takes dZ as the sum hi + lo of two f16 values, which leaves 2^-23
// of each term. f16 rather than X's dtype, since two bf16 values leave 2^-17;
// bf16 rows of X are scaled by 2^-e to f16, every row so that its largest value
// lies in [2^14, 2^15) (row_top_exp_of), and their rows of dZ by 2^e: a row's
// dZ is as large as what the row gives to the tables. (The logits' exponents
// jump from 0 to -17 where a row's largest value falls below 2^-2; rows on
// both sides under one scale lost up to 17 of the 23 bits.) dX has a form of
// its own then: a row of X near zero has no gradient to give to the tables, but
// takes one itself.
// The f16 forms are scaled by powers of two; the results are scaled back in
// fp32 (exact). dLUT's sum over the tokens takes one scale for all, which puts
// the largest row factor, |dloss| 2^e, into [2^14, 2^15): a term keeps 2^-23 of
// itself or 2^-39 of that factor, whichever is more. dX's rows are apart, so
// every token's |dloss| is put there by itself (xent_token_exp) and a softmax
// value down to 2^-28 keeps f16's full precision, however far the tokens'
// weights lie apart. Only f16 X with both gradients shares one form, with
// dLUT's scale: a third one would be written and read for tokens whose dX
// hardly fills f16. bf16 dZ (dX with bf16 tables) needs no scale.
//
// Bound by the matrix tiles. 4096 tokens, three quarters of them scored, 32000
// words of 4096 columns (b = 4, f16): statistics 724 us (1113 TFLOP/s), dZ 794, dX
// 861 (935 TFLOP/s), dLUT 1219, all else 75. 2001 tokens, statistics only: 490 us.
//
// Tokens whose target is ignore_index are left out: the index kernel lists the
// others, and every kernel works on that list with its length read on the
// device. (The few-token kernel computes their logits and drops them.) No value
// of an ignored token's row of X, which may hold anything, reaches a result; its
// loss, lse and dX are zeros.
#pragma once

#include "skm_common.h"
#include "skm_launch.h"

namespace skm {

// at the start of the workspace
struct XentHead {
  int32_t count;    // tokens that have a target
  float scale;      // of dLUT's f16 operands, a power of two, and its inverse
  float inv_scale;
  DxPlan dx;        // ranges of dX's tiles (dx_plan)
};

// exponent of the power of two that puts a value of this magnitude pattern
// into [2^14, 2^15) (0 for zero and what is smaller than fp32's normal values)
__device__ __forceinline__ int scale_exp(uint32_t top) {
  const int e = top >= 0x00800000u ? 14 + 127 - (int)(top >> 23) : 0;
  return e > 126 ? 126 : (e < -112 ? -112 : e);
}
// of a token's dZ as dX's f16 operand
__device__ __forceinline__ int xent_token_exp(float dloss) {
  return scale_exp(__builtin_bit_cast(uint32_t, dloss) & 0x7FFFFFFFu);
}

// ---- pieces of the launchers, one translation unit each --------------------------

// rows of a launch: listed tokens (p.m the most there can be) x p.n weight rows
struct XentGemm {
  const void* X;
  int x_dtype;
  const uint8_t* idx;
  const void* lut;
  int lut_dtype;
  Problem p;
  const int32_t* rows;
  const XentHead* head;
  const int64_t* targets;
  const int32_t* rexp;  // row exponents of X, by token (mixed pair)
  int64_t v0;
  const void* Xp;       // the listed rows in the tables' dtype, in K order (xent_streams)
};
// whether the logit tiles read their activations and indices straight into LDS
// (skm_xent_logits.h), from a copy of the listed rows that xent_rows makes
inline bool xent_streams(const Problem& p) { return p.b == 4 && p.group_cols() % 64 == 0; }
hipError_t xent_stats(const XentGemm& g, float2* part, int64_t stride, float* tlogit, hipStream_t s);
struct XentGradOut {
  const float* lse;
  const float* dloss;
  int64_t V, ld;
  void *hi, *lo, *dxv;  // see EpGrad
  const int32_t* zexp;  // exponents e of dZ's f16 rows, by token (NULL = 0)
  float* rest;          // [listed row] remainder of the target's term in dX's operand
};
hipError_t xent_grad(const XentGemm& g, const XentGradOut& o, hipStream_t s);

// Few tokens (skm_xent_decode.h): 16 per block of the decode kernel, rows of
// X in token order (not listed). part: [token][16-row block]
bool xent_few(const Problem& p);
bool xent_decode_stages(const Problem& p);  // activations in LDS, no row exponents needed
hipError_t xent_few_stats(const XentGemm& g, float2* part, int64_t blocks, float* tlogit, hipStream_t s);
hipError_t xent_few_grad(const XentGemm& g, const XentGradOut& o, const int32_t* pos, hipStream_t s);

}  // namespace skm
