// Small checks of arguments that the entry points share.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "fp8kv_attn.h"

namespace fp8kv {

inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
inline bool strides_ok(const int64_t* s, int n, int64_t unit) {
  for (int i = 0; i < n; ++i)
    if (s[i] < 0 || s[i] % unit) return false;
  return true;
}
// From x to y, in floats (both on their boundary).
inline int64_t floats_between(const float* x, const float* y) {
  return ((int64_t)reinterpret_cast<uintptr_t>(y) - (int64_t)reinterpret_cast<uintptr_t>(x)) / 4;
}
// Finite host scales, or device floats on their boundary.
template <class Args>
inline bool scales_ok(const Args& a) {
  return aligned(a.k_scale_dev, 4) && aligned(a.v_scale_dev, 4) && (a.k_scale_dev || std::isfinite(a.k_scale)) &&
         (a.v_scale_dev || std::isfinite(a.v_scale));
}
inline bool fp8_format(int32_t f) { return f == FP8KV_KV_E4M3 || f == FP8KV_KV_E5M2; }
inline int done(cudaError_t e) { return e == cudaSuccess ? FP8KV_OK : FP8KV_ECUDA; }

}  // namespace fp8kv
