// Cross entropy forward: the instances of the matmul's tiles that end in
// softmax statistics (EpStats).
#include "skm_xent_logits.h"

namespace skm {

namespace {

template <int B, typename TX, typename TL>
hipError_t stats_b(const XentGemm& g, float2* part, int64_t stride, float* tlogit, hipStream_t s) {
  typedef EpStats EP;
  typename EP::Args a;
  a.rows = g.rows;
  a.count = &g.head->count;
  a.targets = g.targets;
  a.v0 = g.v0;
  a.part = part;
  a.stride = stride;
  a.tlogit = tlogit;
  if constexpr (B == 4)
    if (xent_streams(g.p)) return xent_logits_launch<TL, EP, !__is_same(TX, TL)>(g, a, s);
  return gemm_fwd_b<B, TX, TL, EP>((const TX*)g.X, g.idx, (const TL*)g.lut, g.p, a, g.rexp, s);
}

template <typename TX, typename TL>
hipError_t stats_t(const XentGemm& g, float2* part, int64_t stride, float* tlogit, hipStream_t s) {
  if (g.p.b == 2) return stats_b<2, TX, TL>(g, part, stride, tlogit, s);
  if (g.p.b == 3) return stats_b<3, TX, TL>(g, part, stride, tlogit, s);
  return stats_b<4, TX, TL>(g, part, stride, tlogit, s);
}

}  // namespace

hipError_t xent_stats(const XentGemm& g, float2* part, int64_t stride, float* tlogit, hipStream_t s) {
  if (g.x_dtype == DT_F16) return stats_t<half_t, half_t>(g, part, stride, tlogit, s);
  if (g.lut_dtype == DT_F16) return stats_t<bf16_t, half_t>(g, part, stride, tlogit, s);
  return stats_t<bf16_t, bf16_t>(g, part, stride, tlogit, s);
}

}  // namespace skm
