// C ABI of dropout, low-rank adapters and head rotation: argument checks.
// The formulas, layouts and error rules are documented in sketch_matmul.h.
#include "sketch_matmul.h"

#include "skm_abi_util.h"
#include "skm_launch.h"

using namespace skm::abi;

namespace {

// dropout's share p as the kernels take it; false: not a probability
bool dropout_of(double p, const int64_t* seed, skm::Dropout& d) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  d = skm::Dropout{(uint32_t)(p * 65536.0 + 0.5), seed};
  return true;
}

// outputs w[0..nw) against each other and against the inputs
bool any_overlap(const Range* w, int nw, const Range* r, int nr) {
  for (int i = 0; i < nw; ++i) {
    for (int j = 0; j < nr; ++j)
      if (overlap(w[i], r[j])) return true;
    for (int j = i + 1; j < nw; ++j)
      if (overlap(w[i], w[j])) return true;
  }
  return false;
}

// ---- rows of heads -----------------------------------------------------------------------

struct Rows {
  const void* p;
  int64_t ld, width;  // elements from row to row, and of a row
};

Range span(Rows a, int64_t m, int es) { return {a.p, a.p ? ((m - 1) * a.ld + a.width) * es : 0}; }

// whether two sets of m rows share a byte. Rows of one stride may lie between each other's (the q and k columns of
// one buffer); of two strides their whole spans are compared.
bool rows_overlap(Rows a, Rows b, int64_t m, int es) {
  if (!overlap(span(a, m, es), span(b, m, es))) return false;
  if (a.ld != b.ld) return true;
  const int64_t row = a.ld * es;
  int64_t off = (int64_t)((intptr_t)b.p - (intptr_t)a.p) % row;
  if (off < 0) off += row;
  return off < a.width * es || off + b.width * es > row;
}

int check_rotary(int64_t m, int q_heads, int k_heads, int head_dim, int rot_dim, int pairs, int norm, float eps,
                 int x_dtype) {
  if (m < 0 || m >= (int64_t(1) << 31)) return SKM_EINVAL;
  if (q_heads < 1 || q_heads > 65536 || k_heads < 0 || k_heads > 65536) return SKM_EINVAL;
  if (head_dim < 2 || head_dim > skm::kMaxHeadDim || head_dim % 2) return SKM_EINVAL;
  if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2) return SKM_EINVAL;
  if (pairs != SKM_PAIRS_HALVES && pairs != SKM_PAIRS_NEIGHBOURS) return SKM_EINVAL;
  if ((norm != 0 && norm != 1) || (norm && !finite_in(eps, 0.f))) return SKM_EINVAL;
  return valid_dtype(x_dtype) ? SKM_OK : SKM_EUNSUPPORTED;
}

// a side's rows: present, wide enough, within 2^40 elements, aligned to an element
int check_rows(Rows a, int64_t m, int es) {
  if (!a.p || a.ld < a.width || a.ld > (int64_t(1) << 40) / (m > 0 ? m : 1)) return SKM_EINVAL;
  return (uintptr_t)a.p % es ? SKM_EALIGN : SKM_OK;
}

}  // namespace

extern "C" {

int sketch_dropout(const void* X, int x_dtype, const void* residual, int64_t count, double p, const int64_t* seed,
                   void* Y, hipStream_t stream) {
  skm::Dropout d;
  if (count < 0 || count > (int64_t(1) << 40) || !dropout_of(p, seed, d)) return SKM_EINVAL;
  if (!valid_dtype(x_dtype)) return SKM_EUNSUPPORTED;
  if (count == 0) return SKM_OK;
  if (!X || !Y || (d.threshold && !seed)) return SKM_EINVAL;
  if (!aligned16(X) || !aligned16(residual) || !aligned16(Y) || ((uintptr_t)seed & 7u) != 0) return SKM_EALIGN;
  const int64_t bytes = count * elem_bytes(x_dtype);
  const Range w{Y, bytes}, r[3] = {{X, bytes}, {residual, bytes}, {seed, 16}};
  if (any_overlap(&w, 1, r, 3)) return SKM_EALIAS;
  return status_of(skm::launch_dropout(X, x_dtype, residual, count, d, Y, stream));
}

// ---- low-rank adapters ---------------------------------------------------------------------

static int check_adapter(int64_t m, int64_t n, int64_t d, int r, int n_adapters, int most, int dtype) {
  if (m < 0 || m > (int64_t(1) << 22) || n < 1 || n > (int64_t(1) << 24)) return SKM_EINVAL;
  if (d < 32 || d % 32 || d > (int64_t(1) << 20)) return SKM_EINVAL;
  if (m * n > (int64_t(1) << 34) || m * d > (int64_t(1) << 34)) return SKM_EINVAL;
  if (r < 1 || r > skm::kMaxAdapterRank || n_adapters < 1 || n_adapters > most) return SKM_EINVAL;
  return dtype == SKM_F16 || dtype == SKM_BF16 ? SKM_OK : SKM_EUNSUPPORTED;
}

// its gradients' launch has a block of 256 threads per 128 columns of dY and X and chunk of tokens (of 128 at least,
// and one per adapter), fewer than 2^32 threads in all
static int check_adapter_bwd(int64_t m, int64_t n, int64_t d, int r, int n_adapters, int dtype) {
  const int st = check_adapter(m, n, d, r, n_adapters, skm::kMaxGradAdapters, dtype);
  if (st != SKM_OK) return st;
  const int64_t strips = (n + 127) / 128 + (d + 127) / 128, chunks = m / 128 + 1 + (n_adapters < m ? n_adapters : m);
  return strips * chunks < (int64_t(1) << 24) ? SKM_OK : SKM_EINVAL;
}

static skm::AdapterArgs adapter_sizes(int64_t m, int64_t n, int64_t d, int r, int n_adapters, int has_ids) {
  skm::AdapterArgs a{};
  a.m = m;
  a.n = n;
  a.d = d;
  a.r = r;
  a.S = n_adapters;
  a.ids = has_ids ? reinterpret_cast<const int32_t*>(16) : nullptr;  // (its presence alone counts)
  return a;
}

constexpr int kMaxAdapters = 1 << 20;

size_t sketch_adapter_fwd_workspace(int64_t m, int64_t n, int64_t d, int r, int n_adapters, int has_ids,
                                    int has_dropout) {
  if (m < 1 || check_adapter(m, n, d, r, n_adapters, kMaxAdapters, SKM_F16) != SKM_OK) return 0;
  skm::AdapterArgs a = adapter_sizes(m, n, d, r, n_adapters, has_ids);
  a.drop.threshold = has_dropout ? 1 : 0;
  return skm::adapter_fwd_bytes(a);
}

int sketch_adapter_fwd(const void* X, const void* A, const void* B, int dtype, const int32_t* adapter, int n_adapters,
                       const float* scale, const void* base, double p, const int64_t* seed, int64_t m, int64_t n,
                       int64_t d, int r, void* Y, float* H, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  const int st = check_adapter(m, n, d, r, n_adapters, kMaxAdapters, dtype);
  if (st != SKM_OK) return st;
  skm::Dropout drop;
  if (!dropout_of(p, seed, drop)) return SKM_EINVAL;
  if (!A || !B || (m > 0 && (!X || !Y || (drop.threshold && !seed)))) return SKM_EINVAL;
  for (const void* q : {X, A, B, base, (const void*)Y, (const void*)H, (const void*)workspace})
    if (!aligned16(q)) return SKM_EALIGN;
  if (((uintptr_t)adapter & 3u) || ((uintptr_t)scale & 3u) || ((uintptr_t)seed & 7u)) return SKM_EALIGN;
  if (m == 0) return SKM_OK;
  const size_t need =
      sketch_adapter_fwd_workspace(m, n, d, r, n_adapters, adapter != nullptr, drop.threshold != 0);
  if (workspace_bytes < need || (need && !workspace)) return SKM_EWORKSPACE;
  const int64_t S = n_adapters;
  const Range w[3] = {{Y, m * n * 2}, {H, m * r * 4}, {need ? workspace : nullptr, (int64_t)need}};
  // (Y may be the base itself: an element is read before it is written, by the same lane)
  const Range in[7] = {{X, m * d * 2},     {A, S * r * d * 2}, {B, S * n * r * 2}, {adapter, m * 4},
                       {scale, S * 4},     {seed, 16},         {base == Y ? nullptr : base, m * n * 2}};
  if (any_overlap(w, 3, in, 7)) return SKM_EALIAS;
  const skm::AdapterArgs a{X, dtype, A, B, adapter, scale, drop, m, n, d, r, n_adapters};
  return status_of(skm::launch_adapter_fwd(a, base, Y, H, workspace, stream));
}

size_t sketch_adapter_bwd_workspace(int64_t m, int64_t n, int64_t d, int r, int n_adapters, int has_ids, int need_dx,
                                    int need_da, int need_db) {
  if (m < 1 || (!need_dx && !need_da && !need_db)) return 0;
  if (check_adapter_bwd(m, n, d, r, n_adapters, SKM_F16) != SKM_OK) return 0;
  return skm::adapter_bwd_bytes(adapter_sizes(m, n, d, r, n_adapters, has_ids), need_dx != 0, need_da != 0,
                                need_db != 0);
}

int sketch_adapter_bwd(const void* dY, const void* X, const float* H, const void* A, const void* B, int dtype,
                       const int32_t* adapter, int n_adapters, const float* scale, const float* base_dx, double p,
                       const int64_t* seed, int64_t m, int64_t n, int64_t d, int r, void* dX, float* dA, float* dB,
                       int accumulate, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_adapter_bwd(m, n, d, r, n_adapters, dtype);
  if (st != SKM_OK) return st;
  skm::Dropout drop;
  if (!dropout_of(p, seed, drop) || (accumulate != 0 && accumulate != 1)) return SKM_EINVAL;
  if (!A || !B) return SKM_EINVAL;
  if (m > 0 && ((dX || dA || dB) && !dY)) return SKM_EINVAL;
  if (m > 0 && ((dA && !X) || (dB && !H) || ((dX || dA) && drop.threshold && !seed))) return SKM_EINVAL;
  for (const void* q : {dY, X, (const void*)H, A, B, (const void*)base_dx, (const void*)dX, (const void*)dA,
                        (const void*)dB, (const void*)workspace})
    if (!aligned16(q)) return SKM_EALIGN;
  if (((uintptr_t)adapter & 3u) || ((uintptr_t)scale & 3u) || ((uintptr_t)seed & 7u)) return SKM_EALIGN;
  const int64_t S = n_adapters;
  if (m == 0) {
    if (!accumulate && dA) st = status_of(skm::launch_zero_f32(dA, S * r * d, stream));
    if (st == SKM_OK && !accumulate && dB) st = status_of(skm::launch_zero_f32(dB, S * n * r, stream));
    return st;
  }
  if (!dX && !dA && !dB) return SKM_OK;
  const size_t need = sketch_adapter_bwd_workspace(m, n, d, r, n_adapters, adapter != nullptr, dX != nullptr,
                                                   dA != nullptr, dB != nullptr);
  if (workspace_bytes < need || !workspace) return SKM_EWORKSPACE;
  const Range w[4] = {{dX, m * d * 2}, {dA, S * r * d * 4}, {dB, S * n * r * 4}, {workspace, (int64_t)need}};
  const Range in[9] = {{dY, m * n * 2},        {X, m * d * 2},   {H, m * r * 4}, {A, S * r * d * 2}, {B, S * n * r * 2},
                       {adapter, m * 4},       {scale, S * 4},   {seed, 16},     {base_dx, m * d * 4}};
  if (any_overlap(w, 4, in, 9)) return SKM_EALIAS;
  const skm::AdapterArgs a{X, dtype, A, B, adapter, scale, drop, m, n, d, r, n_adapters};
  return status_of(skm::launch_adapter_bwd(a, dY, H, base_dx, dX, dA, dB, accumulate, workspace, stream));
}

// ---- norm and rotation of heads --------------------------------------------------------------

int sketch_rotary_fwd(const void* Q, int64_t ldq, int q_heads, const void* K, int64_t ldk, int k_heads, int x_dtype,
                      const int64_t* positions, const double* inv_freq, const float* q_weight, const float* k_weight,
                      int64_t m, int head_dim, int rot_dim, int pairs, int norm, float eps, void* Qout, int64_t ldqo,
                      void* Kout, int64_t ldko, hipStream_t stream) {
  int st = check_rotary(m, q_heads, k_heads, head_dim, rot_dim, pairs, norm, eps, x_dtype);
  if (st != SKM_OK) return st;
  if (m == 0) return SKM_OK;
  if (!positions || !inv_freq) return SKM_EINVAL;
  const int es = elem_bytes(x_dtype);
  const int64_t qw = (int64_t)q_heads * head_dim, kw = (int64_t)k_heads * head_dim;
  const Rows in[2] = {{Q, ldq, qw}, {K, ldk, kw}}, out[2] = {{Qout, ldqo, qw}, {Kout, ldko, kw}};
  const int sides = k_heads ? 2 : 1;
  for (int i = 0; i < sides; ++i)
    if ((st = check_rows(in[i], m, es)) != SKM_OK || (st = check_rows(out[i], m, es)) != SKM_OK) return st;
  if (((uintptr_t)positions & 7u) || ((uintptr_t)inv_freq & 7u) || !aligned16(q_weight) || !aligned16(k_weight))
    return SKM_EALIGN;
  for (int i = 0; i < sides; ++i) {
    for (int j = 0; j < sides; ++j) {
      // (in place: a head is read whole before its lanes write it)
      const bool same = i == j && out[i].p == in[j].p && out[i].ld == in[j].ld;
      if (!same && rows_overlap(out[i], in[j], m, es)) return SKM_EALIAS;
    }
    const Range o = span(out[i], m, es);
    if (overlap(o, {positions, m * 8}) || overlap(o, {inv_freq, (int64_t)rot_dim * 4}) ||
        (norm && (overlap(o, {q_weight, (int64_t)head_dim * 4}) || overlap(o, {k_weight, (int64_t)head_dim * 4}))))
      return SKM_EALIAS;
  }
  if (sides == 2 && rows_overlap(out[0], out[1], m, es)) return SKM_EALIAS;
  const skm::RotaryArgs a{{Q, nullptr, Qout, ldq, 0, ldqo, norm ? q_weight : nullptr, q_heads},
                          {K, nullptr, Kout, ldk, 0, ldko, norm ? k_weight : nullptr, k_heads},
                          positions, inv_freq, m, head_dim, rot_dim, pairs, norm, eps};
  return status_of(skm::launch_rotary_fwd(a, x_dtype, stream));
}

size_t sketch_rotary_bwd_workspace(int head_dim) {
  return head_dim >= 2 && head_dim <= skm::kMaxHeadDim ? skm::rotary_bwd_part_bytes(head_dim) : 0;
}

int sketch_rotary_bwd(const void* dQ, int64_t lddq, int q_heads, const void* dK, int64_t lddk, int k_heads,
                      int x_dtype, const void* Q, int64_t ldq, const void* K, int64_t ldk, const int64_t* positions,
                      const double* inv_freq, const float* q_weight, const float* k_weight, int64_t m, int head_dim,
                      int rot_dim, int pairs, int norm, float eps, void* dXq, int64_t ldxq, void* dXk, int64_t ldxk,
                      float* dq_weight, float* dk_weight, int accumulate, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
  int st = check_rotary(m, q_heads, k_heads, head_dim, rot_dim, pairs, norm, eps, x_dtype);
  if (st != SKM_OK) return st;
  if (accumulate != 0 && accumulate != 1) return SKM_EINVAL;
  if ((dq_weight || dk_weight) && !norm) return SKM_EINVAL;
  if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(dq_weight) || !aligned16(dk_weight) ||
      !aligned16(workspace) || ((uintptr_t)positions & 7u) || ((uintptr_t)inv_freq & 7u))
    return SKM_EALIGN;
  if (m == 0) {
    if (!accumulate && dq_weight) st = status_of(skm::launch_zero_f32(dq_weight, head_dim, stream));
    if (st == SKM_OK && !accumulate && dk_weight) st = status_of(skm::launch_zero_f32(dk_weight, head_dim, stream));
    return st;
  }
  if (!positions || !inv_freq) return SKM_EINVAL;
  const int es = elem_bytes(x_dtype), sides = k_heads ? 2 : 1;
  const int64_t qw = (int64_t)q_heads * head_dim, kw = (int64_t)k_heads * head_dim;
  const Rows dy[2] = {{dQ, lddq, qw}, {dK, lddk, kw}}, out[2] = {{dXq, ldxq, qw}, {dXk, ldxk, kw}};
  const Rows x[2] = {{norm ? Q : nullptr, ldq, qw}, {norm ? K : nullptr, ldk, kw}};
  for (int i = 0; i < sides; ++i) {
    if ((st = check_rows(dy[i], m, es)) != SKM_OK || (st = check_rows(out[i], m, es)) != SKM_OK) return st;
    if (norm && (st = check_rows(x[i], m, es)) != SKM_OK) return st;
  }
  const size_t need = dq_weight || dk_weight ? sketch_rotary_bwd_workspace(head_dim) : 0;
  if (workspace_bytes < need || (need && !workspace)) return SKM_EWORKSPACE;
  const int64_t wb = (int64_t)head_dim * 4;
  const Range w[3] = {{dq_weight, wb}, {dk_weight, wb}, {need ? workspace : nullptr, (int64_t)need}};
  Range r[8] = {{positions, m * 8}, {inv_freq, (int64_t)rot_dim * 4}, {q_weight, wb}, {k_weight, wb}};
  for (int i = 0; i < 2; ++i) {
    r[4 + 2 * i] = i < sides ? span(dy[i], m, es) : Range{nullptr, 0};
    r[5 + 2 * i] = i < sides ? span(x[i], m, es) : Range{nullptr, 0};
  }
  if (any_overlap(w, 3, r, 8)) return SKM_EALIAS;
  for (int i = 0; i < sides; ++i) {
    const Range o = span(out[i], m, es);
    for (int j = 0; j < 4; ++j)
      if (overlap(o, r[j]) || (j < 3 && overlap(o, w[j]))) return SKM_EALIAS;
    for (int j = 0; j < sides; ++j)
      if (rows_overlap(out[i], dy[j], m, es) || (norm && rows_overlap(out[i], x[j], m, es))) return SKM_EALIAS;
  }
  if (sides == 2 && rows_overlap(out[0], out[1], m, es)) return SKM_EALIAS;
  const skm::RotaryArgs a{{x[0].p, dQ, dXq, ldq, lddq, ldxq, norm ? q_weight : nullptr, q_heads},
                          {x[1].p, dK, dXk, ldk, lddk, ldxk, norm ? k_weight : nullptr, k_heads},
                          positions, inv_freq, m, head_dim, rot_dim, pairs, norm, eps};
  return status_of(
      skm::launch_rotary_bwd(a, x_dtype, dq_weight, dk_weight, accumulate, need ? (float*)workspace : nullptr, stream));
}

}  // extern "C"
