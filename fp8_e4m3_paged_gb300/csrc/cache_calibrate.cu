// Scale calibration: *scale = max(*scale, max |x| / fmax) over the finite
// elements of the new K (V) rows.
//
// The maximum is taken on the elements' magnitude bits (ordered as integers),
// two per 32-bit word with one SIMD maximum, so a 16-byte piece costs four
// AND + maximum pairs and the kernel is bound by HBM (2 bytes per element).
// Infinities and NaNs (bits at or above the type's infinity) show up in the
// running maximum; only a batch that held one is gone through again with them taken out.
// Each CTA ends with one integer atomicMax per stream on the float's bits
// (positive floats order as integers, so the result does not depend on the
// order); x / fmax is monotone, so the largest quotient is the quotient of
// the largest magnitude.
// Measured: 65536 tokens of 8 heads x 128, 268 MB, 39 us: the rate of a plain copy
// (reading alone is a little faster); 64 tokens 2.0 us, a launch.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"
#include "chunk.h"

namespace fp8kv {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // 16-byte pieces in flight per thread

__device__ const int64_t kNoSlots = 0;  // the slot of every token when there is no mapping

template <int DT>
__device__ __forceinline__ uint32_t mag_max(uint32_t m, uint32_t w, bool finite_only) {
  constexpr uint32_t kInf = DT == FP8KV_DTYPE_F16 ? 0x7C00u : 0x7F80u;
  uint32_t x = w & 0x7FFF7FFFu;
  if (finite_only) {
    if ((x & 0xFFFFu) >= kInf) x &= 0xFFFF0000u;
    if ((x >> 16) >= kInf) x &= 0x0000FFFFu;
  }
  return __vmaxu2(m, x);
}

// blockIdx.y: 0 = K, 1 = V.
template <int DT, bool PACKED>
__global__ void __launch_bounds__(kThreads) calibrate_kernel(const fp8kv_calibrate_args a) {
  constexpr uint32_t kInf = DT == FP8KV_DTYPE_F16 ? 0x7C00u : 0x7F80u;
  const bool is_v = blockIdx.y == 1;
  const uint16_t* src = reinterpret_cast<const uint16_t*>(is_v ? a.v : a.k);
  const int64_t st = is_v ? a.v_stride_token : a.k_stride_token, sh = is_v ? a.v_stride_head : a.k_stride_head;
  const int per_head = a.head_dim / 8, per_token = a.num_kv_heads * per_head;
  const int64_t total = (int64_t)a.num_tokens * per_token;
  uint32_t best = 0u;
  // a CTA takes runs of kBatch * kThreads pieces
  for (int64_t i0 = (int64_t)blockIdx.x * (kBatch * kThreads) + threadIdx.x; i0 < total;
       i0 += (int64_t)gridDim.x * (kBatch * kThreads)) {
    uint4 w[kBatch];
    int64_t slot[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      // past the last: the last once more (a load under a condition is waited for on the spot)
      const int64_t i = min(i0 + j * kThreads, total - 1);
      const uint16_t* at;
      if (PACKED) {
        at = src + i * 8;
      } else {
        const int64_t n = i / per_token;
        slot[j] = __ldg((a.slot_mapping ? a.slot_mapping : &kNoSlots) + (a.slot_mapping ? n : 0));
        const int rem = (int)(i - n * per_token), h = rem / per_head;
        at = src + n * st + h * sh + (rem - h * per_head) * 8;
      }
      w[j] = __ldcs(reinterpret_cast<const uint4*>(at));
    }
    if (!PACKED) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (slot[j] < 0) w[j] = make_uint4(0, 0, 0, 0);
    }
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      m = mag_max<DT>(m, w[j].x, false);
      m = mag_max<DT>(m, w[j].y, false);
      m = mag_max<DT>(m, w[j].z, false);
      m = mag_max<DT>(m, w[j].w, false);
    }
    if ((m & 0xFFFFu) >= kInf || (m >> 16) >= kInf) {
      m = 0u;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        m = mag_max<DT>(m, w[j].x, true);
        m = mag_max<DT>(m, w[j].y, true);
        m = mag_max<DT>(m, w[j].z, true);
        m = mag_max<DT>(m, w[j].w, true);
      }
    }
    best = __vmaxu2(best, m);
  }
  uint32_t top = max(best & 0xFFFFu, best >> 16);
  top = __reduce_max_sync(0xffffffffu, top);
  __shared__ uint32_t warp_top[kThreads / 32];
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x < 32) {
    top = threadIdx.x < kThreads / 32 ? warp_top[threadIdx.x] : 0u;
    top = __reduce_max_sync(0xffffffffu, top);
    if (threadIdx.x == 0 && top != 0u) {
      const float x = DT == FP8KV_DTYPE_F16 ? __half2float(__ushort_as_half((unsigned short)top))
                                            : __uint_as_float(top << 16);
      const float q = __fdiv_rn(x, a.kv_format == FP8KV_KV_E5M2 ? 57344.f : 448.f);
      atomicMax(reinterpret_cast<int*>(is_v ? a.v_scale : a.k_scale), __float_as_int(q));
    }
  }
}

}  // namespace

namespace {

template <int DT, bool PACKED>
cudaError_t run(const fp8kv_calibrate_args& a, int64_t total, cudaStream_t st) {
  static ResidentCtas resident;
  int cap = 0;
  const cudaError_t e = resident.get(calibrate_kernel<DT, PACKED>, kThreads, &cap);
  if (e != cudaSuccess) return e;
  const int64_t need = (total + kBatch * kThreads - 1) / (kBatch * kThreads), half = (cap + 1) / 2;
  calibrate_kernel<DT, PACKED><<<dim3((unsigned)(need < half ? need : half), 2), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_calibrate(const fp8kv_calibrate_args& a, cudaStream_t st) {
  // rows that lie side by side need no index arithmetic
  const int64_t D = a.head_dim, row = D * a.num_kv_heads, total = (int64_t)a.num_tokens * row / 8;
  const bool packed = !a.slot_mapping && a.k_stride_head == D && a.v_stride_head == D && a.k_stride_token == row &&
                      a.v_stride_token == row;
  if (a.dtype == FP8KV_DTYPE_F16)
    return packed ? run<FP8KV_DTYPE_F16, true>(a, total, st) : run<FP8KV_DTYPE_F16, false>(a, total, st);
  return packed ? run<FP8KV_DTYPE_BF16, true>(a, total, st) : run<FP8KV_DTYPE_BF16, false>(a, total, st);
}

}  // namespace fp8kv
