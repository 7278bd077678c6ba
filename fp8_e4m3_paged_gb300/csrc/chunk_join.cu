// Joins the partitions of a split chunk attention: per (row, query head)
//
//   M = max_s m_s,  out = v_scale sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s
//
// from the FP32 numerators o_s, maxima m_s (base 2) and sums l_s.  One warp
// per vector, lanes along d (float4 or float2 each); a few MB at most, bound by
// latency and launch.
#include <cstdint>

#include <cuda_runtime.h>

#include "chunk_common.cuh"

namespace fp8kv {
namespace {

constexpr int kJoinThreads = 128;

// 2^x for the weight of a partition that saw something: never 0, so that an
// infinite numerator of a far smaller partition stays infinite (0 * inf).
__device__ __forceinline__ float part_weight(float x) { return exp2f(fmaxf(x, -120.f)); }

template <int D, int DT>
__global__ void __launch_bounds__(kJoinThreads) chunk_join(const ChunkParams p) {
  constexpr int V = D / 32;  // floats per lane
  const int lane = threadIdx.x & 31;
  const int64_t vec = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int row = (int)(vec / p.Hq), h = (int)(vec - (int64_t)row * p.Hq);
  if (row >= p.total_q) return;
  // the request of the row: the number of ends at or below it
  int b = 0;
  for (int i0 = 0; i0 < p.B; i0 += 32) {
    const bool below = i0 + lane < p.B && p.cu_q[i0 + lane + 1] <= row;
    b += __popc(__ballot_sync(0xffffffffu, below));
  }
  if (b >= p.B) return;  // behind the last request
  const ChunkRequest r = chunk_request(p, b);
  if (row < r.row0 || row - r.row0 >= r.n) return;
  const int64_t plane = (int64_t)p.total_q * p.Hq;
  float M = kNoMax;
  for (int s = lane; s < p.S; s += 32) M = fmaxf(M, p.ml[s * plane + vec].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[V] = {};
  float L = 0.f;
  for (int s = 0; s < p.S; ++s) {
    const float2 ml = p.ml[s * plane + vec];
    if (ml.x == kNoMax && ml.y == 0.f) continue;  // saw nothing (a NaN sum is kept)
    const float w = ml.x == M ? 1.f : part_weight(ml.x - M);
    L = fmaf(w, ml.y, L);
    const float* src = p.partial + (s * plane + vec) * D + lane * V;
    float x[V];
    if constexpr (V == 2) {
      *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 4) *reinterpret_cast<float4*>(x + j) = *reinterpret_cast<const float4*>(src + j);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = fmaf(w, x[j], acc[j]);
  }
  const float vs = p.v_scale_dev ? *p.v_scale_dev : p.v_scale;
  const float inv = L == 0.f ? 0.f : vs / L;
  uint32_t o[V / 2];
#pragma unroll
  for (int j = 0; j < V; j += 2) o[j / 2] = L == 0.f ? 0u : pack_out<DT>(acc[j] * inv, acc[j + 1] * inv);
  uint16_t* dst = p.out + row * p.o_st + h * p.o_sh + lane * V;
  if constexpr (V == 2)
    *reinterpret_cast<uint32_t*>(dst) = o[0];
  else if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
  else
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace

cudaError_t launch_chunk_join(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  constexpr int F16 = FP8KV_DTYPE_F16, BF16 = FP8KV_DTYPE_BF16;
  const bool bf = plan->dtype == BF16;
  void (*fn)(const ChunkParams) = nullptr;
  switch (plan->head_dim) {
    case 64: fn = bf ? chunk_join<64, BF16> : chunk_join<64, F16>; break;
    case 128: fn = bf ? chunk_join<128, BF16> : chunk_join<128, F16>; break;
    default: fn = bf ? chunk_join<256, BF16> : chunk_join<256, F16>; break;
  }
  const int64_t n = (int64_t)p.total_q * p.Hq, per = kJoinThreads / 32;
  fn<<<(unsigned)((n + per - 1) / per), kJoinThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8kv
