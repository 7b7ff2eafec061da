// Argument checks shared by the C ABI's files.
#pragma once

#include <cmath>

#include "sketch_matmul.h"

namespace skm {
namespace abi {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem_bytes(int dt) { return dt == SKM_F32 ? 4 : 2; }

inline bool valid_dtype(int dt) { return dt == SKM_F32 || dt == SKM_F16 || dt == SKM_BF16; }

struct Range {
  const void* p;
  int64_t bytes;
};

inline bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? SKM_OK : SKM_EHIP; }

// finite and at least lo
inline bool finite_in(float v, float lo) { return std::isfinite(v) && v >= lo; }

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace abi
}  // namespace skm
