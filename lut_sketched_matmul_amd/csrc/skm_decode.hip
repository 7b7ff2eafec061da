// Decode-sized forward pass for m <= 16 tokens: the plain matmul's instances
// of the kernel in skm_decode.h.
#include "skm_decode.h"

namespace skm {

namespace {

template <int B, int NW, typename TX, typename TL>
hipError_t decode_nw(const TX* X, const uint8_t* idx, const TL* lut, const Problem& p, TX* Y, hipStream_t s,
                     uint32_t magic, const SetArgs& sa) {
  // one table set: stage the activations when all m rows fit. Several sets:
  // each pass stages its own tokens, so it suffices that one row fits (with a
  // single set in use, the m rows then take several passes)
  const bool multi = sa.lut_set && !sa.select;
  const bool xl = decode_stages_activations(p, multi, sa.n_sets,
                                            scaled_pair(__is_same(TX, bf16_t), __is_same(TL, half_t)));
  // Unstaged, one set: from 8 tokens on, the coalesced loads and the LDS
  // turn-around cost less than loading fragments directly (whose cost grows
  // with the distinct token rows a load touches); below, the direct loads.
  const bool xt = !xl && !multi && p.m >= DEC_XT_MIN_M;
  typedef EpDecodeStore<TX> EP;
  if (p.units() % 4 != 0)
    return xl ? decode_launch<B, NW, TX, TL, true, true, false, EP>(X, idx, lut, p, {Y}, s, magic, sa)
              : (xt ? decode_launch<B, NW, TX, TL, true, false, true, EP>(X, idx, lut, p, {Y}, s, magic, sa)
                    : decode_launch<B, NW, TX, TL, true, false, false, EP>(X, idx, lut, p, {Y}, s, magic, sa));
  return xl ? decode_launch<B, NW, TX, TL, false, true, false, EP>(X, idx, lut, p, {Y}, s, magic, sa)
            : (xt ? decode_launch<B, NW, TX, TL, false, false, true, EP>(X, idx, lut, p, {Y}, s, magic, sa)
                  : decode_launch<B, NW, TX, TL, false, false, false, EP>(X, idx, lut, p, {Y}, s, magic, sa));
}

template <int B, typename TX, typename TL>
hipError_t decode_b(const TX* X, const uint8_t* idx, const TL* lut, const Problem& p, TX* Y, hipStream_t s,
                    const SetArgs& sa) {
  const uint32_t ug = (uint32_t)(p.group_cols() / 32);
  // u / ug == umulhi(u, magic) for u * ug < 2^32; ug == 1 is passed as 0
  const uint32_t magic = ug == 1 ? 0u : (uint32_t)((((uint64_t)1) << 32) / ug + 1);
  // Few 16-row blocks (one per CU or less): 16 waves per block for more loads
  // in flight. Many blocks: 8 waves so two or more blocks share a CU and one
  // block's start-up latency hides behind another's work.
  const int64_t blocks = (p.n + DEC_ROWS - 1) / DEC_ROWS;
  const int nw = blocks <= 384 ? 16 : 8;
  if (nw == 16) return decode_nw<B, 16>(X, idx, lut, p, Y, s, magic, sa);
  return decode_nw<B, 8>(X, idx, lut, p, Y, s, magic, sa);
}

template <typename TX, typename TL>
hipError_t decode_t(const TX* X, const uint8_t* idx, const TL* lut, const Problem& p, TX* Y, hipStream_t s,
                    const SetArgs& sa) {
  switch (p.b) {
    case 2: return decode_b<2>(X, idx, lut, p, Y, s, sa);
    case 3: return decode_b<3>(X, idx, lut, p, Y, s, sa);
    default: return decode_b<4>(X, idx, lut, p, Y, s, sa);
  }
}

hipError_t decode_dispatch(const void* X, int x_dtype, const uint8_t* idx, const void* lut, int lut_dtype,
                           const Problem& p, void* Y, hipStream_t s, const SetArgs& sa) {
  if (x_dtype == DT_F16 && lut_dtype == DT_F16)
    return decode_t((const half_t*)X, idx, (const half_t*)lut, p, (half_t*)Y, s, sa);
  if (x_dtype == DT_BF16 && lut_dtype == DT_F16)
    return decode_t((const bf16_t*)X, idx, (const half_t*)lut, p, (bf16_t*)Y, s, sa);
  if (x_dtype == DT_F16 && lut_dtype == DT_BF16)
    return decode_t((const half_t*)X, idx, (const bf16_t*)lut, p, (half_t*)Y, s, sa);
  return decode_t((const bf16_t*)X, idx, (const bf16_t*)lut, p, (bf16_t*)Y, s, sa);
}

}  // namespace

int decode_max_m() { return 16; }

bool decode_stages_activations(const Problem& p, bool multi, int n_sets, bool scaled) {
  // the prescaled multi-set decode always stages (it finds the exponents of
  // the staged rows itself). One set: up to 32768 elements, or, below the
  // token count from which the LDS turn-around runs (staging 72-96 KB per
  // block measured slower than that), up to 49152 when the grid has at most
  // one 16-row block per CU (more LDS per block then costs no occupancy) and
  // tables, activations, 16 partial tiles and the magnitude slots fit in
  // 160 KB.
  if (p.m * p.d <= DEC_XL_MAX) return true;
  if (multi) return (n_sets > 1 || scaled) && p.d <= DEC_XL_MAX;
  const int64_t T = p.b == 2 ? 16 : p.k();
  const int64_t lds = p.gpr * T * 256 + p.m * p.d * 2 + 16 * 1024 + 17 * 16 * 4;
  return p.m < DEC_XT_MIN_M && p.m * p.d <= DEC_XL_MAX1 && (p.n + DEC_ROWS - 1) / DEC_ROWS <= 256 &&
         lds <= 160 * 1024;
}

bool decode_multi_supported(const Problem& p, bool scaled) {
  // the prescaled pair stages its activations in the one-pass-per-set kernel
  // (rows of at most 32768 columns); the set-interleaved kernel (m >= 2)
  // finds its row exponents without staging, and takes every set count when
  // the entries per row fit two cells (a set count above 8 needs that)
  const int64_t E = (int64_t)p.gpr << p.b;
  return decode_supported(p) && (!scaled || p.d <= DEC_XL_MAX || (p.m >= 2 && E <= (p.m > 8 ? 128 : 224)));
}

bool decode_supported(const Problem& p) {
  const int T = p.b == 2 ? 16 : p.k();
  // the magic-number division by units-per-group is exact while U * UG < 2^32
  return p.m >= 1 && p.m <= 16 && (int64_t)p.gpr * T <= DEC_MAX_ENTRIES && p.d <= (int64_t(1) << 20);
}

hipError_t launch_decode(const void* X, int x_dtype, const uint8_t* idx, const void* lut, int lut_dtype,
                         const Problem& p, void* Y, const int32_t* rexp, hipStream_t s) {
  SetArgs sa;
  sa.rexp = rexp;
  return decode_dispatch(X, x_dtype, idx, lut, lut_dtype, p, Y, s, sa);
}

hipError_t launch_decode_multi(const void* X, int x_dtype, const uint8_t* idx, const void* luts, int lut_dtype,
                               const int32_t* lut_set, int n_sets, const Problem& p, void* Y, hipStream_t s) {
  // one set: the single-set decode (every token on set 0); one token: the
  // single-set decode on that token's set (found on the device), when it
  // needs no row exponents from a workspace; else set-interleaved tables
  // whenever they apply; otherwise one pass per set in use
  const bool scaled = x_dtype == DT_BF16 && lut_dtype == DT_F16;
  if (n_sets == 1 && !scaled) return decode_dispatch(X, x_dtype, idx, luts, lut_dtype, p, Y, s, SetArgs{});
  if (p.m == 1 && (!scaled || decode_stages_activations(p, false, 1, true))) {
    SetArgs one;
    one.lut_set = lut_set;
    one.select = true;
    one.n_sets = n_sets;
    one.set_stride = p.n * p.gpr * p.k();
    return decode_dispatch(X, x_dtype, idx, luts, lut_dtype, p, Y, s, one);
  }
  if (decode_sets_supported(p, n_sets, scaled))
    return launch_decode_sets(X, x_dtype, idx, luts, lut_dtype, lut_set, n_sets, p, Y, s);
  SetArgs sa;
  sa.lut_set = lut_set;
  sa.n_sets = n_sets;
  sa.set_stride = p.n * p.gpr * p.k();
  return decode_dispatch(X, x_dtype, idx, luts, lut_dtype, p, Y, s, sa);
}

}  // namespace skm
