// 8-bit activation checkpoints: writing (k_act_quant), reading back
// (k_act_dequant) and the backward of a sketched layer whose X is one
// (launch_bwd_ckpt). The format is in skm_quant.h.
//
// Rows are whole blocks of 32 columns, so a matrix is one flat run of blocks
// and each kernel a stream: a lane takes 8 columns (four lanes per block, whose
// largest magnitude two quad permutes find), kept in registers between the
// maximum and the rounding, so every value is read once.
// Bound by memory: 8192 x 11008 bf16 written in 49 us and read back in 41 (5.6 and
// 6.7 TB/s of the bytes each has to move; a large copy reaches 5.15 to 6.2). Non-temporal
// stores write 8 % faster, but the product that reads the codes next misses them.
#include "skm_launch.h"
#include "skm_quant.h"

namespace skm {

namespace {

template <typename T>
__global__ void __launch_bounds__(256) k_act_quant(const T* __restrict__ X, int64_t chunks, int8_t* __restrict__ codes,
                                                   uint8_t* __restrict__ scales) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;  // chunks is a multiple of 4: quads stay whole
  u32x4 w[sizeof(T) / 2];
#pragma unroll
  for (int q = 0; q < (int)sizeof(T) / 2; ++q) w[q] = reinterpret_cast<const u32x4*>(X + c * 8)[q];
  uint32_t s;
  *reinterpret_cast<u32x2*>(codes + c * 8) = ckpt_of<T>(w, s);
  if ((threadIdx.x & 3) == 0) scales[c >> 2] = (uint8_t)s;
}

// chunks .. total - 1 of X are written as zeros
template <typename T>
__global__ void __launch_bounds__(256) k_act_dequant(const int8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales, int64_t chunks,
                                                     int64_t total, T* __restrict__ X) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= total) return;
  float v[8] = {};
  if (c < chunks) ckpt_unpack8(*reinterpret_cast<const u32x2*>(codes + c * 8), scales[c >> 2], v);
  store8<T>(X + c * 8, v);
}

// rows of n 16-bit values to rows of ld (a multiple of 8), zeros past n and in
// rows m .. cap - 1
__global__ void __launch_bounds__(256) k_pad_rows(const uint16_t* __restrict__ src, int64_t m, int64_t n, int64_t cap,
                                                  int64_t ld, uint16_t* __restrict__ dst) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (q >= cap * (ld / 8)) return;
  const int64_t r = q / (ld / 8), j = q % (ld / 8) * 8;
  uint32_t v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = r < m && j + k < n ? src[r * n + j + k] : 0u;
  *reinterpret_cast<u32x4*>(dst + r * ld + j) =
      u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

// out = sum of the ranges' parts, in order; four values per thread
__global__ void __launch_bounds__(256) k_sum_ranges(const float* __restrict__ part, int ranges, int64_t count,
                                                    float* __restrict__ out) {
  const int64_t q = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (q >= count) return;
  f32x4 s = *reinterpret_cast<const f32x4*>(part + q);
  for (int k = 1; k < ranges; ++k) s += *reinterpret_cast<const f32x4*>(part + (int64_t)k * count + q);
  *reinterpret_cast<f32x4*>(out + q) = s;
}

template <typename T>
hipError_t dequant_to(const int8_t* codes, const uint8_t* scales, int64_t count, int64_t total, void* X,
                      hipStream_t s) {
  hipLaunchKernelGGL(k_act_dequant<T>, dim3((unsigned)((total / 8 + 255) / 256)), dim3(256), 0, s, codes, scales,
                     count / 8, total / 8, (T*)X);
  return hipGetLastError();
}
hipError_t dequant(const int8_t* codes, const uint8_t* scales, int64_t count, int64_t total, void* X, int x_dtype,
                   hipStream_t s) {
  if (x_dtype == DT_F32) return dequant_to<float>(codes, scales, count, total, X, s);
  if (x_dtype == DT_F16) return dequant_to<half_t>(codes, scales, count, total, X, s);
  return dequant_to<bf16_t>(codes, scales, count, total, X, s);
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: X in io_dtype, padded to whole 32-token steps, and 16 zero bytes;
// dY with 16-byte aligned rows when its own are not; row exponents of dY; the
// ranges' dX; partial dLUT tables
struct CkptPlan {
  int64_t cap, ld;
  bool pad;
  DxRanges r;
  size_t x, y, rexp, dx, part, bytes;
};
CkptPlan ckpt_plan(const Problem& p, int io_dtype, int lut_dtype, bool need_dx, bool need_dlut) {
  CkptPlan f;
  f.cap = (p.m + 31) / 32 * 32;
  f.pad = p.n % 8 != 0;
  f.ld = (p.n + 7) / 8 * 8;
  f.r = dx_ranges(p);
  size_t o = 0;
  auto take = [&](bool on, size_t bytes) {
    const size_t at = o;
    if (on) o += up256(bytes);
    return at;
  };
  f.x = take(need_dlut, ((size_t)f.cap * (size_t)p.d + 8) * 2);
  f.y = take(f.pad, (size_t)f.cap * (size_t)f.ld * 2);
  f.rexp = take(need_dx && scaled_pair(io_dtype == DT_BF16, lut_dtype == DT_F16), (size_t)p.m * 4);
  f.dx = take(need_dx && f.r.count > 1, (size_t)f.r.count * (size_t)p.m * (size_t)p.d * 4);
  f.part = take(need_dlut, dlut_partial_bytes(p));
  f.bytes = o;
  return f;
}

}  // namespace

hipError_t launch_act_quant(const void* X, int x_dtype, int64_t count, int8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t chunks = count / 8;
  const dim3 grid((unsigned)((chunks + 255) / 256));
  if (x_dtype == DT_F32)
    hipLaunchKernelGGL(k_act_quant<float>, grid, dim3(256), 0, s, (const float*)X, chunks, codes, scales);
  else if (x_dtype == DT_F16)
    hipLaunchKernelGGL(k_act_quant<half_t>, grid, dim3(256), 0, s, (const half_t*)X, chunks, codes, scales);
  else
    hipLaunchKernelGGL(k_act_quant<bf16_t>, grid, dim3(256), 0, s, (const bf16_t*)X, chunks, codes, scales);
  return hipGetLastError();
}

hipError_t launch_act_dequant(const int8_t* codes, const uint8_t* scales, int64_t count, void* X, int x_dtype,
                              hipStream_t s) {
  return dequant(codes, scales, count, count, X, x_dtype, s);
}

size_t bwd_ckpt_bytes(const Problem& p, int io_dtype, int lut_dtype, bool need_dx, bool need_dlut) {
  return ckpt_plan(p, io_dtype, lut_dtype, need_dx, need_dlut).bytes;
}

// The checkpoint is read back once, into the operand type (its values are
// exact there), and the table gradient's tiles stream that copy from memory
// straight into LDS. Converting inside the tiles instead would repeat the
// conversion in each of the n / 128 row blocks, about 20 vector instructions
// per operand fragment that feeds two MFMAs.
hipError_t launch_bwd_ckpt(const void* dY, const int8_t* codes, const uint8_t* scales, int io_dtype,
                           const uint8_t* idx, const void* lut, int lut_dtype, const Problem& p, float* dX,
                           float* dLUT, int accumulate, void* ws, hipStream_t s) {
  const CkptPlan f = ckpt_plan(p, io_dtype, lut_dtype, dX != nullptr, dLUT != nullptr);
  char* base = static_cast<char*>(ws);
  hipError_t e = hipSuccess;
  const void* y = dY;
  if (f.pad) {
    const int64_t chunks = f.cap * (f.ld / 8);
    hipLaunchKernelGGL(k_pad_rows, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, s, (const uint16_t*)dY, p.m,
                       p.n, f.cap, f.ld, (uint16_t*)(base + f.y));
    y = base + f.y;
    e = hipGetLastError();
  }
  if (e == hipSuccess && dX) {
    int32_t* rexp = nullptr;
    if (scaled_pair(io_dtype == DT_BF16, lut_dtype == DT_F16)) {
      rexp = reinterpret_cast<int32_t*>(base + f.rexp);
      e = launch_row_exp(y, p.m, f.ld, rexp, s);
    }
    const bool ranges = f.r.count > 1;
    float* parts = reinterpret_cast<float*>(base + f.dx);
    if (e == hipSuccess)
      e = launch_dx_piece(y, io_dtype, idx, lut, lut_dtype, p, ranges ? parts : dX, rexp, nullptr, f.ld, 0, f.r,
                          nullptr, 0, s);
    if (e == hipSuccess && ranges) {
      const int64_t count = p.m * p.d;
      hipLaunchKernelGGL(k_sum_ranges, dim3((unsigned)((count / 4 + 255) / 256)), dim3(256), 0, s, parts, f.r.count,
                         count, dX);
      e = hipGetLastError();
    }
  }
  if (e != hipSuccess || !dLUT) return e;
  char* x = base + f.x;
  const int64_t count = p.m * p.d, padded = f.cap * p.d;
  e = dequant(codes, scales, count, padded + 8, x, io_dtype, s);
  if (e != hipSuccess) return e;
  const DlutPiece q{nullptr, f.ld, nullptr, f.pad || p.m % 32 == 0 ? nullptr : x + padded * 2};
  return launch_dlut_piece(y, nullptr, x, io_dtype, idx, p, dLUT, accumulate, reinterpret_cast<float*>(base + f.part),
                           q, s);
}

}  // namespace skm
