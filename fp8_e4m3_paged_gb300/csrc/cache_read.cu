// Cache read: rows of the paged FP8 cache back as fp16, bf16 or FP32.
//
//   out = round(fp32(dec(byte)) * scale)
//
// dec() is exact in fp16, the product is one FP32 rounding, the output type a
// second one (none for FP32).  Bound by HBM: one byte in and 2 or 4 out per
// element.  A CTA takes a run of output rows; its first threads find each
// row's request (binary search of cu_len) and place once, then
// all threads move 16-byte pieces, K and V of the same place together.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk_common.cuh"
#include "internal.h"

namespace fp8kv {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;               // 16-byte pieces per thread and stream
constexpr int kMaxRows = kThreads;      // rows of a CTA

// 16 FP8 bytes * scale -> 16 output elements.
template <int DT, int FMT>
__device__ __forceinline__ void expand16(const uint4& w, float scale, void* dst) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  float f[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t lo, hi;
    fp8x4_to_f16<FMT>(in[j], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    f[4 * j] = a.x * scale;
    f[4 * j + 1] = a.y * scale;
    f[4 * j + 2] = b.x * scale;
    f[4 * j + 3] = b.y * scale;
  }
  if constexpr (DT == FP8KV_DTYPE_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      reinterpret_cast<float4*>(dst)[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      reinterpret_cast<uint4*>(dst)[j] =
          make_uint4(pack_out<DT>(f[8 * j], f[8 * j + 1]), pack_out<DT>(f[8 * j + 2], f[8 * j + 3]),
                     pack_out<DT>(f[8 * j + 4], f[8 * j + 5]), pack_out<DT>(f[8 * j + 6], f[8 * j + 7]));
  }
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const fp8kv_cache_read_args a, int rows_per_cta) {
  constexpr int ES = DT == FP8KV_DTYPE_F32 ? 4 : 2;
  __shared__ int64_t s_k[kMaxRows], s_v[kMaxRows];  // byte offset of the row, -1 bad place, -2 not written
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * rows_per_cta;
  const int n = (int)min((int64_t)rows_per_cta, a.total - row0);
  if (tid < n) {
    const int row = (int)row0 + tid;
    // the last request that begins at or below the row
    int lo = 0, hi = a.batch;  // cu_len[lo] <= row < cu_len[hi], if the row is covered
    const int first = __ldg(a.cu_len), last = __ldg(a.cu_len + a.batch);
    int64_t ko = -2, vo = -2;
    if (row >= first && row < last) {
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu_len + mid) <= row)
          lo = mid;
        else
          hi = mid;
      }
      const int c0 = __ldg(a.cu_len + lo);
      const int64_t t = (int64_t)row - c0 + (a.start ? __ldg(a.start + lo) : 0);
      ko = vo = -1;
      if (t >= 0 && t < (int64_t)a.max_blocks * a.page_size) {
        const int64_t page = t / a.page_size;
        const int slot = (int)(t - page * a.page_size);
        const int64_t blk = __ldg(a.block_table + lo * a.block_table_stride + page);
        if (blk >= 0 && blk < a.num_kv_blocks) {
          ko = blk * a.kc_stride_block + slot * a.kc_stride_token;
          vo = blk * a.vc_stride_block + slot * a.vc_stride_token;
        }
      }
      if (ko == -1 && a.status) set_status(a.status, FP8KV_STATUS_BAD_BLOCK);
    }
    s_k[tid] = ko;
    s_v[tid] = vo;
  }
  if (blockIdx.x == 0 && a.status) {
    // one CTA checks the lengths; whatever they are, rows stay in [0, total)
    for (int i = tid; i <= a.batch; i += kThreads) {
      const int x = __ldg(a.cu_len + i);
      if (x < (i ? __ldg(a.cu_len + i - 1) : 0) || x > a.total) set_status(a.status, FP8KV_STATUS_BAD_LEN);
    }
  }
  const float ks = a.k_scale_dev ? *a.k_scale_dev : a.k_scale;
  const float vs = a.v_scale_dev ? *a.v_scale_dev : a.v_scale;
  __syncthreads();
  const int per_head = a.head_dim / 16, per_row = a.num_kv_heads * per_head;
  const int64_t items = (int64_t)n * per_row;
  for (int64_t i0 = tid; i0 < items; i0 += kItems * kThreads) {
    uint4 kx[kItems], vx[kItems];
    int row[kItems], h[kItems], c[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int64_t i = i0 + j * kThreads;
      row[j] = -1;
      if (i >= items) continue;
      row[j] = (int)(i / per_row);
      const int rem = (int)(i - (int64_t)row[j] * per_row);
      h[j] = rem / per_head;
      c[j] = rem - h[j] * per_head;
      const int64_t ko = s_k[row[j]], vo = s_v[row[j]];
      kx[j] = vx[j] = make_uint4(0, 0, 0, 0);
      if (ko == -2) row[j] = -1;
      if (ko >= 0) {
        kx[j] = __ldcs(reinterpret_cast<const uint4*>(a.k_cache + ko + h[j] * a.kc_stride_head + c[j] * 16));
        vx[j] = __ldcs(reinterpret_cast<const uint4*>(a.v_cache + vo + h[j] * a.vc_stride_head + c[j] * 16));
      }
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      if (row[j] < 0) continue;
      const bool gone = s_k[row[j]] < 0;  // +0.0 whatever the scale's sign
      const int64_t r = row0 + row[j];
      expand16<DT, FMT>(kx[j], gone ? 1.f : ks,
                        reinterpret_cast<uint8_t*>(a.k_out) +
                            (r * a.ko_stride_token + h[j] * a.ko_stride_head + c[j] * 16) * ES);
      expand16<DT, FMT>(vx[j], gone ? 1.f : vs,
                        reinterpret_cast<uint8_t*>(a.v_out) +
                            (r * a.vo_stride_token + h[j] * a.vo_stride_head + c[j] * 16) * ES);
    }
  }
}

}  // namespace

cudaError_t launch_cache_read(const fp8kv_cache_read_args& a, cudaStream_t st) {
  constexpr int E4 = FP8KV_KV_E4M3, E5 = FP8KV_KV_E5M2;
  constexpr int F16 = FP8KV_DTYPE_F16, BF16 = FP8KV_DTYPE_BF16, F32 = FP8KV_DTYPE_F32;
  void (*fn)(const fp8kv_cache_read_args, int);
  const bool e5 = a.kv_format == E5;
  if (a.dtype == F16)
    fn = e5 ? cache_read_kernel<F16, E5> : cache_read_kernel<F16, E4>;
  else if (a.dtype == BF16)
    fn = e5 ? cache_read_kernel<BF16, E5> : cache_read_kernel<BF16, E4>;
  else
    fn = e5 ? cache_read_kernel<F32, E5> : cache_read_kernel<F32, E4>;
  const int64_t per_row = (int64_t)a.num_kv_heads * (a.head_dim / 16);
  int64_t rows = kItems * kThreads / per_row;  // one pass of the CTA
  rows = rows < 1 ? 1 : rows > kMaxRows ? kMaxRows : rows;
  const int64_t grid = (a.total + rows - 1) / rows;
  fn<<<(unsigned)grid, kThreads, 0, st>>>(a, (int)rows);
  return cudaGetLastError();
}

}  // namespace fp8kv
