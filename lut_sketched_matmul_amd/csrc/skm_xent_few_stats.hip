// Cross entropy forward of few tokens: the decode kernel's instances that end
// in softmax statistics.
#include "skm_xent_decode.h"

namespace skm {

namespace {

template <typename TX, typename TL>
hipError_t few_t(const XentGemm& g, float2* part, int64_t blocks, float* tlogit, hipStream_t s) {
  typedef EpDecodeStats EP;
  const typename EP::Args a{g.targets, part, blocks, tlogit, 0};
  if (g.p.b == 2) return xent_decode<2, TX, TL, EP>(g, a, s);
  if (g.p.b == 3) return xent_decode<3, TX, TL, EP>(g, a, s);
  return xent_decode<4, TX, TL, EP>(g, a, s);
}

}  // namespace

hipError_t xent_few_stats(const XentGemm& g, float2* part, int64_t blocks, float* tlogit, hipStream_t s) {
  if (g.x_dtype == DT_F16) return few_t<half_t, half_t>(g, part, blocks, tlogit, s);
  if (g.lut_dtype == DT_F16) return few_t<bf16_t, half_t>(g, part, blocks, tlogit, s);
  return few_t<bf16_t, bf16_t>(g, part, blocks, tlogit, s);
}

}  // namespace skm
