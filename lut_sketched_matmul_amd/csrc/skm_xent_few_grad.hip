// Cross entropy backward of few tokens: the decode kernel's instances that end
// in the logits' gradient.
#include "skm_xent_decode.h"

namespace skm {

namespace {

template <typename TX, typename TL>
hipError_t few_t(const XentGemm& g, const XentGradOut& o, const int32_t* pos, hipStream_t s) {
  typedef EpDecodeGrad<TX, TL> EP;
  const typename EP::Args a{pos,        g.head, g.targets, o.lse, o.dloss,      o.zexp,        o.V, g.v0,
                            o.ld,       0,      (half_t*)o.hi,   (half_t*)o.lo, (TL*)o.dxv, o.rest};
  if (g.p.b == 2) return xent_decode<2, TX, TL, EP>(g, a, s);
  if (g.p.b == 3) return xent_decode<3, TX, TL, EP>(g, a, s);
  return xent_decode<4, TX, TL, EP>(g, a, s);
}

}  // namespace

hipError_t xent_few_grad(const XentGemm& g, const XentGradOut& o, const int32_t* pos, hipStream_t s) {
  if (g.x_dtype == DT_F16) return few_t<half_t, half_t>(g, o, pos, s);
  if (g.lut_dtype == DT_F16) return few_t<bf16_t, half_t>(g, o, pos, s);
  return few_t<bf16_t, bf16_t>(g, o, pos, s);
}

}  // namespace skm
