// The query and key heads between a projection and attention: the norm of each
// head and its position's rotation in one pass, forward and backward.
//   r  = 1 / sqrt(mean_head(x^2) + eps), z = x r w          (without a norm z = x)
//   (y_a, y_b) = (z_a c - z_b s, z_a s + z_b c), c, s = cos, sin(position f_i)
// for the pairs (a, b) = (i, i + rot / 2) or (2 i, 2 i + 1), i < rot / 2; columns
// from rot on pass. Backward, g = the rotation's transpose (s -> -s) of dy:
//   dw = sum g x r,  dx = r g w - x r^3 mean_head(g w x)
//
// Angles are fp64 products, reduced to [-pi/4, pi/4] in fp64 (two-term pi/2), so
// a far position loses nothing; the sine and cosine of the rest are Taylor sums in
// fp32, once per token and pair, shared through LDS by all of the token's heads.
// A lane keeps both members of V pairs (two vectors of a head), so rotation needs
// no exchange; a head's sums go over its 1 to 64 lanes. V = 8 (16-byte vectors of a
// 16-bit type) where the heads and rows allow it, else V = 1.
//
// Bound by memory: 8192 tokens, 72 heads of 128, bf16 with norm 59 us (5.1 TB/s); backward of 4096 tokens, 64 heads,
// f16, 44 us (4.6 TB/s) and 4.6 us for the blocks' sums; one token's 40 heads 5.3 us. Fetching the next heads early
// measured the same or worse (59.8 and 48 us: more registers, fewer waves).
//
// The weight gradients: each block keeps its lanes' sums in registers over the
// tokens it walks, adds them up in LDS, and k_rotary_reduce adds the blocks'
// rows in block order (deterministic, no atomics).
#include <type_traits>

#include "skm_launch.h"
#include "skm_quant.h"

namespace skm {

namespace {

constexpr int THREADS = 256;
constexpr int64_t kBwdBlocks = 768;  // of the backward at most: three per CU run at once (512 blocks: 46 us, 768: 44, 1024: 49)
constexpr int MAX_TRIG = kMaxHeadDim / 2;  // (token, pair) angles a block holds

// cos and sin of pos * freq
__device__ __forceinline__ void angle_of(int64_t pos, double freq, float& c, float& s) {
  const double a = (double)pos * freq;
  const double k = rint(a * 0.63661977236758134308);   // 2 / pi
  double r = fma(-k, 1.5707963267948965580, a);         // pi / 2 to 53 bits
  r = fma(-k, 6.1232339957367660359e-17, r);            // and what is left of it
  const float x = (float)r, q = x * x;
  // Taylor sums; on |x| <= pi / 4 the first term left out is below 2^-28 of the sum
  const float sn = x * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f);
  const float cs = fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const int n = (int)(int64_t)(k - 4.0 * floor(k * 0.25));  // quarter turns, 0..3
  const float u = n & 1 ? cs : sn, v = n & 1 ? sn : cs;
  s = n & 2 ? -u : u;
  c = n == 1 || n == 2 ? -v : v;
}

template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&v)[V]) {
  if constexpr (V == 8) load8<T>(p, v);
  else v[0] = to_f32(p[0]);
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 8) store8<T>(p, v);
  else p[0] = from_f32<T>(v[0]);
}

// sum over the L lanes of a head (L a power of two), in every one of them
template <int L>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < L; o *= 2) v += __shfl_xor(v, o);
  return v;
}

struct Side {
  const void* x;
  const void* dy;
  void* y;
  int64_t ldx, lddy, ldy;  // in elements
  const float* w;          // NULL = ones
  int heads;
};

struct RotaryGrid {
  Side q, k;
  const int64_t* pos;
  const double* freq;
  int64_t m;
  int dh, rot, neighbours, norm;
  float eps;
  int tokens;  // a block's tokens at a time
  float* part;  // weight gradients of the blocks [grid][2][dh], NULL = none
};

// columns of slot s (V pairs): first vector, second vector, first angle
template <int V>
__device__ __forceinline__ void slot_cols(const RotaryGrid& a, int s, int& c0, int& c1, bool& turns) {
  turns = s * V < a.rot / 2;
  const bool halves = turns && !a.neighbours;
  c0 = halves ? V * s : 2 * V * s;
  c1 = halves ? a.rot / 2 + V * s : c0 + V;
}

// turn (or turn back) the pairs of a slot; cs / sn: the token's angles of this slot
template <int V, bool BACK>
__device__ __forceinline__ void turn(float (&u)[V], float (&v)[V], const float* cs, const float* sn, bool neighbours) {
  if constexpr (V == 8) {
    float c[8], s[8];
    load8<float>(cs, c);
    load8<float>(sn, s);
    if (BACK) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = -s[j];
    }
    if (!neighbours) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = u[j] * c[j] - v[j] * s[j];
        v[j] = u[j] * s[j] + v[j] * c[j];
        u[j] = x;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x = u[2 * j] * c[j] - u[2 * j + 1] * s[j];
        u[2 * j + 1] = u[2 * j] * s[j] + u[2 * j + 1] * c[j];
        u[2 * j] = x;
        x = v[2 * j] * c[4 + j] - v[2 * j + 1] * s[4 + j];
        v[2 * j + 1] = v[2 * j] * s[4 + j] + v[2 * j + 1] * c[4 + j];
        v[2 * j] = x;
      }
    }
  } else {
    const float c = cs[0], s = BACK ? -sn[0] : sn[0];
    const float x = u[0] * c - v[0] * s;
    v[0] = u[0] * s + v[0] * c;
    u[0] = x;
  }
}

// V pairs a lane and slot, L lanes a head, NS slots a lane
template <typename T, int V, int L, int NS, bool BWD>
__device__ __forceinline__ void side_units(const RotaryGrid& a, const Side& p, int64_t t0, int nt, int u0, int u1,
                                           const float* cs, const float* sn, float (&dw)[NS][2][V]) {
  const int lane = threadIdx.x % L, rank = threadIdx.x / L;
  constexpr int UNITS = THREADS / L;
  const int slots = a.dh / (2 * V), half = a.rot / 2;
  float w[NS][2][V];
  int c0[NS], c1[NS];
  bool turns[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int s = lane + L * i;
    slot_cols<V>(a, s < slots ? s : 0, c0[i], c1[i], turns[i]);
    turns[i] = turns[i] && s < slots;  // (a lane behind the last slot has no angles)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[i][0][j] = p.w ? p.w[c0[i] + j] : 1.f;
      w[i][1][j] = p.w ? p.w[c1[i] + j] : 1.f;
    }
  }
  const int total = nt * p.heads;
  u1 = u1 < total ? u1 : total;
  for (int u = u0 + rank; u < u1; u += UNITS) {
    const int tk = u / p.heads, h = u - tk * p.heads;
    const int64_t t = t0 + tk;
    float x[NS][2][V], g[NS][2][V];
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const bool in = lane + L * i < slots;
      if (!BWD || a.norm) {
        const T* row = (const T*)p.x + t * p.ldx + (int64_t)h * a.dh;
        load_v<T, V>(row + c0[i], x[i][0]);
        load_v<T, V>(row + c1[i], x[i][1]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][0][j] = x[i][1][j] = 0.f;
      }
      if (BWD) {
        const T* row = (const T*)p.dy + t * p.lddy + (int64_t)h * a.dh;
        load_v<T, V>(row + c0[i], g[i][0]);
        load_v<T, V>(row + c1[i], g[i][1]);
      }
      if (in) {
#pragma unroll
        for (int j = 0; j < V; ++j) sq += x[i][0][j] * x[i][0][j] + x[i][1][j] * x[i][1][j];
      }
    }
    float r = 1.f;
    if (a.norm) r = 1.f / sqrtf(head_sum<L>(sq) / (float)a.dh + a.eps);
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int s = lane + L * i;
        if (a.norm) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            x[i][0][j] = x[i][0][j] * r * w[i][0][j];
            x[i][1][j] = x[i][1][j] * r * w[i][1][j];
          }
        }
        if (turns[i]) turn<V, false>(x[i][0], x[i][1], cs + tk * half + s * V, sn + tk * half + s * V, a.neighbours);
        T* out = (T*)p.y + t * p.ldy + (int64_t)h * a.dh;
        if (s < slots) {
          store_v<T, V>(out + c0[i], x[i][0]);
          store_v<T, V>(out + c1[i], x[i][1]);
        }
      }
    } else {
      float gx = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int s = lane + L * i;
        if (turns[i]) turn<V, true>(g[i][0], g[i][1], cs + tk * half + s * V, sn + tk * half + s * V, a.neighbours);
        if (a.norm && s < slots) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              dw[i][q][j] += g[i][q][j] * (x[i][q][j] * r);
              g[i][q][j] *= w[i][q][j];
              gx += g[i][q][j] * x[i][q][j];
            }
        }
      }
      float f = 0.f;
      if (a.norm) f = head_sum<L>(gx) / (float)a.dh * r * r * r;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int s = lane + L * i;
        if (a.norm) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < V; ++j) g[i][q][j] = g[i][q][j] * r - x[i][q][j] * f;
        }
        T* out = (T*)p.y + t * p.ldy + (int64_t)h * a.dh;
        if (s < slots) {
          store_v<T, V>(out + c0[i], g[i][0]);
          store_v<T, V>(out + c1[i], g[i][1]);
        }
      }
    }
  }
}

template <typename T, int V, int L, int NS, bool BWD>
__global__ __launch_bounds__(THREADS) void k_rotary(RotaryGrid a) {
  __shared__ __align__(16) float cs[MAX_TRIG], sn[MAX_TRIG];
  __shared__ float sums[BWD ? THREADS * 2 * V : 1];
  const int half = a.rot / 2;
  float dwq[NS][2][V], dwk[NS][2][V];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) dwq[i][0][j] = dwq[i][1][j] = dwk[i][0][j] = dwk[i][1][j] = 0.f;
  // the block's share of the units (token, head) of a's tokens
  const int uq = a.tokens * a.q.heads, uk = a.tokens * a.k.heads;
  constexpr int UNITS = THREADS / L;
  const int pq = ((uq + UNITS - 1) / UNITS + gridDim.y - 1) / gridDim.y * UNITS;
  const int pk = ((uk + UNITS - 1) / UNITS + gridDim.y - 1) / gridDim.y * UNITS;
  const int yq = (int)blockIdx.y * pq, yk = (int)(gridDim.y - 1 - blockIdx.y) * pk;
  const int64_t groups = (a.m + a.tokens - 1) / a.tokens;
  for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    const int64_t t0 = grp * a.tokens;
    const int nt = (int)(a.m - t0 < a.tokens ? a.m - t0 : a.tokens);
    __syncthreads();  // (the last group's angles are still read)
    for (int i = threadIdx.x; i < nt * half; i += THREADS) {
      const int tk = i / half;
      angle_of(a.pos[t0 + tk], a.freq[i - tk * half], cs[i], sn[i]);
    }
    __syncthreads();
    side_units<T, V, L, NS, BWD>(a, a.q, t0, nt, yq, yq + pq, cs, sn, dwq);
    if (a.k.heads) side_units<T, V, L, NS, BWD>(a, a.k, t0, nt, yk, yk + pk, cs, sn, dwk);
  }
  if constexpr (BWD) {
    if (!a.part) return;
    const int slots = a.dh / (2 * V);
    float* row = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.dh;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int j = 0; j < V; ++j)
            sums[(q * V + j) * THREADS + threadIdx.x] = side ? dwk[i][q][j] : dwq[i][q][j];
        __syncthreads();
        // value e of the 2 V of lane l: the sum over the block's THREADS / L ranks, in rank order
        for (int e = threadIdx.x; e < 2 * V * L; e += THREADS) {
          const int l = e % L, v = e / L, s = l + L * i;
          if (s < slots) {
            float t = 0.f;
            for (int k = 0; k < UNITS; ++k) t += sums[v * THREADS + k * L + l];
            int c0, c1;
            bool turns;
            slot_cols<V>(a, s, c0, c1, turns);
            row[side * a.dh + (v < V ? c0 + v : c1 + v - V)] = t;
          }
        }
      }
    }
  }
}

// dw[c] (+)= sum over the blocks' rows: four columns a block, 64 threads a column, each every 64th row
__global__ __launch_bounds__(256) void k_rotary_reduce(const float* __restrict__ part, int rows, int dh, float* dqw,
                                                       float* dkw, int accumulate) {
  __shared__ float sh[64][4];
  const int x = threadIdx.x & 3, y = threadIdx.x >> 2;
  const int c = blockIdx.x * 4 + x, side = blockIdx.y;
  float* out = side ? dkw : dqw;
  float t = 0.f;
  if (c < dh) {
#pragma unroll 8
    for (int r = y; r < rows; r += 64) t += part[((int64_t)r * 2 + side) * dh + c];
  }
  sh[y][x] = t;
  __syncthreads();
  if (y || c >= dh || !out) return;
  t = 0.f;
  for (int k = 0; k < 64; ++k) t += sh[k][x];
  out[c] = accumulate ? out[c] + t : t;
}

bool vector_rows(const RotaryArgs& a, int es, bool bwd) {
  if (a.dh % 16 || a.rot % 16) return false;
  auto ok = [&](const RotarySide& s) {
    if (!s.heads) return true;
    auto one = [&](const void* p, int64_t ld) { return ((uintptr_t)p & 15u) == 0 && ld * es % 16 == 0; };
    return (!s.x || one(s.x, s.ldx)) && one(s.y, s.ldy) && (!bwd || one(s.dy, s.lddy));
  };
  return ok(a.q) && ok(a.k);
}

// tokens a block holds the angles of, and its grid
struct Plan {
  int tokens;
  unsigned gx, gy;
};
Plan plan_of(const RotaryArgs& a, int L, bool bwd) {
  const int half = a.rot / 2;
  int t = half < 256 ? 256 / half : 1;
  if (t > 16) t = 16;
  // Few tokens: one at a time, its heads over several blocks. (Enough tokens
  // for two blocks per CU: their angles are worth sharing.)
  while (t > 1 && (a.m + t - 1) / t < 512) t /= 2;
  const int64_t groups = (a.m + t - 1) / t;
  const int64_t units = (int64_t)t * a.q.heads, steps = (units * L + THREADS - 1) / THREADS;
  int64_t gy = 1;
  if (groups < 512) {
    gy = 512 / groups;
    if (gy > steps) gy = steps;
  }
  const int64_t most = bwd ? (kBwdBlocks / gy > 1 ? kBwdBlocks / gy : 1) : 65536;
  return Plan{t, (unsigned)(groups < most ? groups : most), (unsigned)gy};
}

template <typename T, bool BWD>
hipError_t rotary_t(const RotaryArgs& a, float* dqw, float* dkw, int accumulate, float* part, hipStream_t s) {
  auto side = [](const RotarySide& p) { return Side{p.x, p.dy, p.y, p.ldx, p.lddy, p.ldy, p.w, p.heads}; };
  auto go = [&](auto v, auto l, auto ns) {
    constexpr int V = decltype(v)::value, L = decltype(l)::value, NS = decltype(ns)::value;
    const Plan g = plan_of(a, L, BWD);
    RotaryGrid r{side(a.q), side(a.k), a.pos, a.freq, a.m, a.dh, a.rot, a.neighbours, a.norm, a.eps, g.tokens, part};
    hipLaunchKernelGGL((k_rotary<T, V, L, NS, BWD>), dim3(g.gx, g.gy), dim3(THREADS), 0, s, r);
    hipError_t e = hipGetLastError();
    if (!BWD || e != hipSuccess || !part) return e;
    hipLaunchKernelGGL(k_rotary_reduce, dim3((unsigned)((a.dh + 3) / 4), 2), dim3(256), 0, s, part,
                       (int)(g.gx * g.gy), a.dh, dqw, dkw, accumulate);
    return hipGetLastError();
  };
  std::integral_constant<int, 1> one;
  if (vector_rows(a, (int)sizeof(T), BWD)) {
    std::integral_constant<int, 8> v;
    const int n = a.dh / 16;
    if (n <= 1) return go(v, std::integral_constant<int, 1>{}, one);
    if (n <= 2) return go(v, std::integral_constant<int, 2>{}, one);
    if (n <= 4) return go(v, std::integral_constant<int, 4>{}, one);
    if (n <= 8) return go(v, std::integral_constant<int, 8>{}, one);
    if (n <= 16) return go(v, std::integral_constant<int, 16>{}, one);
    if (n <= 32) return go(v, std::integral_constant<int, 32>{}, one);
    return go(v, std::integral_constant<int, 64>{}, one);
  }
  const int n = a.dh / 2;
  if (n <= 16) return go(one, std::integral_constant<int, 16>{}, one);
  std::integral_constant<int, 64> l;
  if (n <= 64) return go(one, l, one);
  if (n <= 128) return go(one, l, std::integral_constant<int, 2>{});
  if (n <= 256) return go(one, l, std::integral_constant<int, 4>{});
  return go(one, l, std::integral_constant<int, 8>{});
}

}  // namespace

size_t rotary_bwd_part_bytes(int64_t dh) { return (size_t)kBwdBlocks * 2 * (size_t)dh * 4; }

hipError_t launch_rotary_fwd(const RotaryArgs& a, int x_dtype, hipStream_t s) {
  if (x_dtype == DT_F32) return rotary_t<float, false>(a, nullptr, nullptr, 0, nullptr, s);
  if (x_dtype == DT_F16) return rotary_t<half_t, false>(a, nullptr, nullptr, 0, nullptr, s);
  return rotary_t<bf16_t, false>(a, nullptr, nullptr, 0, nullptr, s);
}

hipError_t launch_rotary_bwd(const RotaryArgs& a, int x_dtype, float* dqw, float* dkw, int accumulate, float* part,
                             hipStream_t s) {
  if (x_dtype == DT_F32) return rotary_t<float, true>(a, dqw, dkw, accumulate, part, s);
  if (x_dtype == DT_F16) return rotary_t<half_t, true>(a, dqw, dkw, accumulate, part, s);
  return rotary_t<bf16_t, true>(a, dqw, dkw, accumulate, part, s);
}

}  // namespace skm
