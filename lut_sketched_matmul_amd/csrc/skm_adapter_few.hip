// The adapters' forward for a few tokens in one launch (skm_adapter.h): one block
// takes one token and 512 columns and computes all of h_t for itself. A_s is then
// read by every block, from the L2 after the first, which costs less than a second
// launch as long as the adapters are small and the tokens few (few_tokens below).
//
// h: a wave takes two or four ranks at a time, a lane eight columns of 512, products in
// fp32 on the vector ALU. y: a thread takes a column, whose ranks are consecutive;
// the first 16 are on their way while h is computed.
#include <type_traits>

#include "skm_adapter.h"

namespace skm {
namespace adapt {

namespace {

constexpr int FEW_WAVES = 8, THREADS = 64 * FEW_WAVES, COLS = THREADS;  // a column a thread

// eight ranks from k0 on of column c, zeros past the rank (rows aligned when r % 8 == 0)
template <typename T>
__device__ __forceinline__ u32x4 ranks_of(const T* B, int64_t c, int r, int k0, bool aligned) {
  const T* p = B + c * r + k0;
  if (aligned) return *reinterpret_cast<const u32x4*>(p);
  return load_some(p, r - k0);
}

// NR: ranks a wave takes at a time
template <typename T, int NR>
__global__ __launch_bounds__(THREADS) void k_adapt_few(const T* __restrict__ X, const T* __restrict__ A,
                                                       const T* __restrict__ B, const int32_t* __restrict__ ids, int S,
                                                       const float* __restrict__ scale, int64_t n, int64_t d, int r,
                                                       const T* base, T* out, float* __restrict__ H) {
  __shared__ float h[kMaxAdapterRank];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.y, c = (int64_t)blockIdx.x * COLS + threadIdx.x;
  const int id = ids ? ids[t] : 0;
  const bool has = id >= 0 && id < S;
  const float y = base && c < n ? to_f32(base[t * n + c]) : 0.f;
  if (!has) {
    for (int k = threadIdx.x; H && blockIdx.x == 0 && k < r; k += THREADS) H[t * r + k] = 0.f;
    if (base != out && c < n) out[t * n + c] = from_f32<T>(y);
    return;
  }
  const T* b = B + (int64_t)id * n * r;
  const bool aligned = r % 8 == 0;
  u32x4 w[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) w[g] = 8 * g < r ? ranks_of(b, c < n ? c : n - 1, r, 8 * g, aligned) : kZero4;

  const T* a = A + (int64_t)id * r * d;
  const T* x = X + t * d;
  for (int k0 = NR * wave; k0 < r; k0 += NR * FEW_WAVES) {
    float acc[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) acc[i] = 0.f;
#pragma unroll 2
    for (int64_t c = 8 * lane; c < d; c += 512) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(x + c);
      u32x4 u[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i)
        u[i] = *reinterpret_cast<const u32x4*>(a + (int64_t)(k0 + i < r ? k0 + i : k0) * d + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xv = unpack<T>(v[j >> 1], j & 1);
#pragma unroll
        for (int i = 0; i < NR; ++i) acc[i] = fmaf(xv, unpack<T>(u[i][j >> 1], j & 1), acc[i]);
      }
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2)
#pragma unroll
      for (int i = 0; i < NR; ++i) acc[i] += __shfl_xor(acc[i], o);
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (lane == i && k0 + i < r) {
        h[k0 + i] = acc[i];
        if (H && blockIdx.x == 0) H[t * r + k0 + i] = acc[i];
      }
  }
  __syncthreads();

  if (c >= n) return;
  float sum = 0.f;
  for (int k0 = 0; k0 < r; k0 += 8) {
    const u32x4 v = k0 == 0 ? w[0] : (k0 == 8 ? w[1] : ranks_of(b, c, r, k0, aligned));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k0 + e < r) sum = fmaf(unpack<T>(v[e >> 1], e & 1), h[k0 + e], sum);
  }
  out[t * n + c] = from_f32<T>(y + (scale ? scale[id] : 1.f) * sum);
}

}  // namespace

// Where this form is the faster one: what the blocks read of A in all, and what the eight XCDs' L2s have to fetch of it
// (each its own copy of every adapter in use). In a graph, this form / two launches, f16:
//   4096 -> 4096, rank 16, 8 adapters: 1 token 4.9 / 8.1 us, 32 tokens 5.4 / 9.9 (34 MB read, 8 fetched)
//   8192 -> 28672, rank 16, 8 adapters: 8 tokens 10.8 / 13.4 (115 MB, 16), 16 tokens 16.9 / 15.2 (230 MB, 16)
//   4096 -> 11008, rank 16, 64 adapters: 32 tokens 12.1 / 14.4 (92 MB, 34), 64 tokens 19.1 / 15.1 (185 MB, 67)
//   4096 -> 4096, rank 32, 64 adapters: 16 tokens 10.7 / 13.3 (34 MB, 34), 32 tokens 15.4 / 13.8 (67 MB, 67)
//   4096 -> 4096, rank 64, 8 adapters: 1 token 11.8 / 12.3, 8 tokens 15.9 / 14.5 (34 MB, 34)
bool few_tokens(const AdapterArgs& a) {
  if (a.m > 128 || a.r > 32 || a.drop.threshold) return false;
  const int64_t one = a.r * a.d * 2, wide = (a.n + COLS - 1) / COLS, S = a.ids ? a.S : 1;
  return a.m * wide * one <= (int64_t(1) << 27) &&
         (S < a.m ? S : a.m) * (wide < 8 ? wide : 8) * one <= (int64_t(34) << 20);
}

hipError_t launch_few(const AdapterArgs& a, const void* base, void* Y, float* H, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + COLS - 1) / COLS), (unsigned)a.m);
  auto go = [&](auto t, auto nr) {
    typedef typename decltype(t)::type T;
    hipLaunchKernelGGL((k_adapt_few<T, decltype(nr)::value>), grid, dim3(THREADS), 0, s, (const T*)a.X, (const T*)a.A,
                       (const T*)a.B, a.ids, a.ids ? a.S : 1, a.scale, a.n, a.d, a.r, (const T*)base, (T*)Y, H);
    return hipGetLastError();
  };
  auto with_ranks = [&](auto t) {
    return a.r <= 2 * FEW_WAVES ? go(t, std::integral_constant<int, 2>{}) : go(t, std::integral_constant<int, 4>{});
  };
  return a.dtype == DT_F16 ? with_ranks(dtype_of<DT_F16>{}) : with_ranks(dtype_of<DT_BF16>{});
}

}  // namespace adapt
}  // namespace skm
