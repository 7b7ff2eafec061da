// Cross entropy backward: the instances of the matmul's tiles that end in the
// logits' gradient (EpGrad).
#include "skm_xent_logits.h"

namespace skm {

namespace {

template <int B, typename TX, typename TL>
hipError_t grad_b(const XentGemm& g, const XentGradOut& o, hipStream_t s) {
  typedef EpGrad<TX, TL> EP;
  typename EP::Args a;
  a.rows = g.rows;
  a.count = &g.head->count;
  a.targets = g.targets;
  a.v0 = g.v0;
  a.lse = o.lse;
  a.dloss = o.dloss;
  a.head = g.head;
  a.zexp = o.zexp;
  a.V = o.V;
  a.ld = o.ld;
  a.hi = (half_t*)o.hi;
  a.lo = (half_t*)o.lo;
  a.dxv = (TL*)o.dxv;
  a.rest = o.rest;
  if constexpr (B == 4)
    if (xent_streams(g.p)) return xent_logits_launch<TL, EP, !__is_same(TX, TL)>(g, a, s);
  return gemm_fwd_b<B, TX, TL, EP>((const TX*)g.X, g.idx, (const TL*)g.lut, g.p, a, g.rexp, s);
}

template <typename TX, typename TL>
hipError_t grad_t(const XentGemm& g, const XentGradOut& o, hipStream_t s) {
  if (g.p.b == 2) return grad_b<2, TX, TL>(g, o, s);
  if (g.p.b == 3) return grad_b<3, TX, TL>(g, o, s);
  return grad_b<4, TX, TL>(g, o, s);
}

}  // namespace

hipError_t xent_grad(const XentGemm& g, const XentGradOut& o, hipStream_t s) {
  if (g.x_dtype == DT_F16) return grad_t<half_t, half_t>(g, o, s);
  if (g.lut_dtype == DT_F16) return grad_t<bf16_t, half_t>(g, o, s);
  return grad_t<bf16_t, bf16_t>(g, o, s);
}

}  // namespace skm
