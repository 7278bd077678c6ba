// Cache read: rows of the paged FP8 cache back as fp16, bf16 or FP32.
//
//   out = round(fp32(dec(byte)) * scale)
//
// dec() is exact in fp16, the product is one FP32 rounding, the output type a
// second one (none for FP32).  Bound by HBM: one byte in and 2 or 4 out per
// element.  Resident CTAs walk tiles of output rows; each row's request
// (binary search of cu_len) and place is found by one thread, for the next
// tile while the current tile's bytes are on their way, so that the chain of
// dependent loads costs nothing.  All threads then move items of 16 output bytes
// (8 or 4 elements), K and V of the same place together: a store instruction of
// 16 bytes out of every 32 would write half sectors.
// Measured: 80000 rows of 8 heads x 128 to fp16, 493 MB in and out, 82 us: 6.0 TB/s,
// 90 % of what a plain copy reaches; three short requests 3.9 us (the launch and the
// chain lengths -> block table -> bytes).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk_common.cuh"
#include "internal.h"

namespace fp8kv {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;               // items per thread and stream in flight
constexpr int kMaxRows = kThreads;      // rows of a tile

// The FP8 bytes of one item (8 for the 16-bit types, 4 for FP32).
template <int DT>
struct Item {
  using Bytes = uint2;
};
template <>
struct Item<FP8KV_DTYPE_F32> {
  using Bytes = uint32_t;
};

template <int FMT>
__device__ __forceinline__ void scaled4(uint32_t w, float scale, float (&f)[4]) {
  uint32_t lo, hi;
  fp8x4_to_f16<FMT>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  f[0] = a.x * scale;
  f[1] = a.y * scale;
  f[2] = b.x * scale;
  f[3] = b.y * scale;
}

// FP8 bytes * scale -> 16 bytes of output elements.
template <int DT, int FMT>
__device__ __forceinline__ uint4 expand(const typename Item<DT>::Bytes& w, float scale) {
  float f[4];
  if constexpr (DT == FP8KV_DTYPE_F32) {
    scaled4<FMT>(w, scale, f);
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    float g[4];
    scaled4<FMT>(w.x, scale, f);
    scaled4<FMT>(w.y, scale, g);
    return make_uint4(pack_out<DT>(f[0], f[1]), pack_out<DT>(f[2], f[3]), pack_out<DT>(g[0], g[1]),
                      pack_out<DT>(g[2], g[3]));
  }
}

// Byte offsets (K, V) of an output row's source: -1 no place (a zero row), -2
// not covered by any request (not written).
__device__ __forceinline__ void find_row(const fp8kv_cache_read_args& a, int row, int64_t& ko, int64_t& vo) {
  ko = vo = -2;
  const int first = __ldg(a.cu_len), last = __ldg(a.cu_len + a.batch);
  if (row < first || row >= last) return;
  // the last request that begins at or below the row
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu_len + mid) <= row)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t t = (int64_t)row - __ldg(a.cu_len + lo) + (a.start ? __ldg(a.start + lo) : 0);
  ko = vo = -1;
  if (t >= 0 && t < (int64_t)a.max_blocks * a.page_size) {
    const int page = (int)(t / a.page_size), slot = (int)(t - (int64_t)page * a.page_size);
    const int64_t blk = __ldg(a.block_table + lo * a.block_table_stride + page);
    if (blk >= 0 && blk < a.num_kv_blocks) {
      ko = blk * a.kc_stride_block + slot * a.kc_stride_token;
      vo = blk * a.vc_stride_block + slot * a.vc_stride_token;
    }
  }
  if (ko == -1 && a.status) set_status(a.status, FP8KV_STATUS_BAD_BLOCK);
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads, 4) cache_read_kernel(const __grid_constant__ fp8kv_cache_read_args a,
                                                              int rows_per_tile) {
  using Bytes = typename Item<DT>::Bytes;
  constexpr int E = sizeof(Bytes), ES = 16 / E;  // elements of an item, bytes of one
  __shared__ int64_t s_k[2][kMaxRows], s_v[2][kMaxRows];
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && a.status) {
    // one CTA checks the lengths; whatever they are, rows stay in [0, total)
    for (int i = tid; i <= a.batch; i += kThreads) {
      const int x = __ldg(a.cu_len + i);
      if (x < (i ? __ldg(a.cu_len + i - 1) : 0) || x > a.total) set_status(a.status, FP8KV_STATUS_BAD_LEN);
    }
  }
  const float ks = a.k_scale_dev ? *a.k_scale_dev : a.k_scale;
  const float vs = a.v_scale_dev ? *a.v_scale_dev : a.v_scale;
  const int per_head = a.head_dim / E, per_row = a.num_kv_heads * per_head;
  const int64_t step = (int64_t)gridDim.x * rows_per_tile;
  auto place = [&](int64_t row0, int buf) {
    if (tid < rows_per_tile && row0 + tid < a.total) find_row(a, (int)(row0 + tid), s_k[buf][tid], s_v[buf][tid]);
  };
  int64_t row0 = (int64_t)blockIdx.x * rows_per_tile;
  place(row0, 0);
  __syncthreads();
  for (int buf = 0; row0 < a.total; row0 += step, buf ^= 1) {
    const int n = (int)min((int64_t)rows_per_tile, a.total - row0);
    const int64_t items = (int64_t)n * per_row;
    bool placed = false;
    for (int64_t i0 = 0; i0 < items; i0 += kItems * kThreads) {
      Bytes kx[kItems], vx[kItems];
      int row[kItems], h[kItems], c[kItems];
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        const int64_t i = min(i0 + j * kThreads + tid, items - 1);  // past the last: read again, not written
        row[j] = (int)(i / per_row);
        const int rem = (int)(i - (int64_t)row[j] * per_row);
        h[j] = rem / per_head;
        c[j] = rem - h[j] * per_head;
        // rows without a place read the pool's first one (a load under a condition is waited for on the spot)
        const int64_t ko = max(s_k[buf][row[j]], (int64_t)0), vo = max(s_v[buf][row[j]], (int64_t)0);
        kx[j] = __ldcs(reinterpret_cast<const Bytes*>(a.k_cache + ko + h[j] * a.kc_stride_head + c[j] * E));
        vx[j] = __ldcs(reinterpret_cast<const Bytes*>(a.v_cache + vo + h[j] * a.vc_stride_head + c[j] * E));
      }
      if (!placed) place(row0 + step, buf ^ 1);
      placed = true;
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        const int64_t at = s_k[buf][row[j]];
        if (at == -2 || i0 + j * kThreads + tid >= items) continue;
        const bool gone = at < 0;  // +0.0 whatever the scale's sign
        if (gone) kx[j] = vx[j] = Bytes{};
        const int64_t r = row0 + row[j];
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.k_out) +
                                        (r * a.ko_stride_token + h[j] * a.ko_stride_head + c[j] * E) * ES),
               expand<DT, FMT>(kx[j], gone ? 1.f : ks));
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.v_out) +
                                        (r * a.vo_stride_token + h[j] * a.vo_stride_head + c[j] * E) * ES),
               expand<DT, FMT>(vx[j], gone ? 1.f : vs));
      }
    }
    __syncthreads();
  }
}

}  // namespace

namespace {

template <int DT, int FMT>
cudaError_t run(const fp8kv_cache_read_args& a, cudaStream_t st) {
  static ResidentCtas resident;
  int cap = 0;
  const cudaError_t e = resident.get(cache_read_kernel<DT, FMT>, kThreads, &cap);
  if (e != cudaSuccess) return e;
  constexpr int E = sizeof(typename Item<DT>::Bytes);
  const int64_t per_row = (int64_t)a.num_kv_heads * (a.head_dim / E);
  int64_t rows = kItems * kThreads / per_row;  // one pass of the CTA
  rows = rows < 1 ? 1 : rows > kMaxRows ? kMaxRows : rows;
  const int64_t tiles = (a.total + rows - 1) / rows;
  cache_read_kernel<DT, FMT><<<(unsigned)(tiles < cap ? tiles : cap), kThreads, 0, st>>>(a, (int)rows);
  return cudaGetLastError();
}

template <int DT>
cudaError_t pick(const fp8kv_cache_read_args& a, cudaStream_t st) {
  return a.kv_format == FP8KV_KV_E5M2 ? run<DT, FP8KV_KV_E5M2>(a, st) : run<DT, FP8KV_KV_E4M3>(a, st);
}

}  // namespace

cudaError_t launch_cache_read(const fp8kv_cache_read_args& a, cudaStream_t st) {
  switch (a.dtype) {
    case FP8KV_DTYPE_F16: return pick<FP8KV_DTYPE_F16>(a, st);
    case FP8KV_DTYPE_BF16: return pick<FP8KV_DTYPE_BF16>(a, st);
    default: return pick<FP8KV_DTYPE_F32>(a, st);
  }
}

}  // namespace fp8kv
