// Joins the partitions of a split chunk attention: per (row, query head)
//
//   M = max_s m_s,  out = v_scale sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s
//
// from the FP32 numerators o_s, maxima m_s (base 2) and sums l_s; lanes along
// d.  A few MB for decode steps, where launch and latency bound it; for long
// chunks the numerators' bytes do (65536 vectors x D 128 in 4 partitions, 151 MB in and
// out: 37 us from a cold cache, 4.0 TB/s).
#include <cstdint>

#include <cuda_runtime.h>

#include "chunk_common.cuh"
#include "dependent.cuh"

namespace fp8kv {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// A CTA's warps are split over vectors and partitions: `ways` warps per vector
// (a power of two) take every ways-th partition each and meet in shared
// memory.  Loads of four partitions are in flight at a time.
// TREE: all rows of a request see the same positions, so its partitions that hold any are
// known, and the others' places are not read.
template <int D, int DT, bool TREE>
__global__ void __launch_bounds__(kJoinThreads) chunk_join(const __grid_constant__ ChunkParams p, const int ways) {
  constexpr int V = D / 32;  // floats per lane
  constexpr int kAhead = 4;
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int way = warp & (ways - 1);
  const int64_t vec = (int64_t)blockIdx.x * (kJoinWarps / ways) + warp / ways;
  const int row = (int)(vec / p.Hq), h = (int)(vec - (int64_t)row * p.Hq);
  bool live = row < p.total_q;
  int S = p.S, U = 0, light = 0;
  if (live) {
    // whether some request has the row among its (clamped) new tokens
    live = false;
    for (int i0 = 0; i0 < p.B && !live; i0 += 32) {
      bool here = false;
      if (i0 + lane < p.B) {
        const ChunkRequest r = chunk_request(p, i0 + lane);
        here = row >= r.row0 && row - r.row0 < r.n;
        if (TREE && here) {
          U = chunk_span<true>(p, r, 0, 0).U;
          light = r.n * p.G <= kChunkTileTokens;
        }
      }
      const uint32_t who = __ballot_sync(0xffffffffu, here);
      live = who != 0u;
      if (TREE && live) {
        U = __shfl_sync(0xffffffffu, U, __ffs(who) - 1);
        light = __shfl_sync(0xffffffffu, light, __ffs(who) - 1);
      }
    }
  }
  if (TREE) {
    wait_for_previous_kernel();
    // (the kernels round partitions up to whole steps: no fewer than these)
    int per = max(1, min((U + p.parts - 1) / p.parts, p.max_part));
    if (p.per_head > 0) per = share_tiles<true>(__ldcg(p.share), light) * kChunkTileTokens;
    S = min(p.S, max(1, (U + per - 1) / per));
  }
  float acc[V] = {};
  float M = kNoMax, L = 0.f;
  if (live) {
    const int64_t plane = (int64_t)p.total_q * p.Hq;
    for (int s = way + ways * lane; s < S; s += 32 * ways) M = fmaxf(M, p.ml[s * plane + vec].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int s0 = way; s0 < S; s0 += kAhead * ways) {
      float2 ml[kAhead];
      float x[kAhead][V];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t at = min(s0 + i * ways, S - 1) * plane + vec;  // past the last: loaded, not used
        ml[i] = p.ml[at];
        const float* src = p.partial + at * D + lane * V;
        if constexpr (V == 2) {
          *reinterpret_cast<float2*>(x[i]) = *reinterpret_cast<const float2*>(src);
        } else {
#pragma unroll
          for (int j = 0; j < V; j += 4)
            *reinterpret_cast<float4*>(x[i] + j) = *reinterpret_cast<const float4*>(src + j);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s0 + i * ways >= S || !part_written(ml[i])) continue;  // (x is stale)
        const float w = part_weight(ml[i].x, M);
        L = fmaf(w, ml[i].y, L);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(w, x[i][j], acc[j]);
      }
    }
  }
  if (ways > 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) s_acc[warp][lane * V + j] = acc[j];
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = L;
    }
    __syncthreads();
    if (way != 0 || !live) return;
    float T = kNoMax;
    for (int w = 0; w < ways; ++w) T = fmaxf(T, s_m[warp + w]);
    L = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int w = 0; w < ways; ++w) {
      const float a = part_weight(s_m[warp + w], T);
      L = fmaf(a, s_l[warp + w], L);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = fmaf(a, s_acc[warp + w][lane * V + j], acc[j]);
    }
  } else if (!live) {
    return;
  }
  const float vs = p.v_scale_dev ? *p.v_scale_dev : p.v_scale;
  const float inv = vs / L;
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

template <bool TREE>
cudaError_t launch(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  constexpr int F16 = FP8KV_DTYPE_F16, BF16 = FP8KV_DTYPE_BF16;
  const bool bf = plan->dtype == BF16;
  void (*fn)(const ChunkParams, int) = nullptr;
  switch (plan->head_dim) {
    case 64: fn = bf ? chunk_join<64, BF16, TREE> : chunk_join<64, F16, TREE>; break;
    case 128: fn = bf ? chunk_join<128, BF16, TREE> : chunk_join<128, F16, TREE>; break;
    default: fn = bf ? chunk_join<256, BF16, TREE> : chunk_join<256, F16, TREE>; break;
  }
  // one warp per vector, more of them while the GPU has idle SMs and each still has partitions
  const int64_t n = (int64_t)p.total_q * p.Hq;
  int ways = 1;
  while (ways < kJoinWarps && 2 * ways <= p.S && n * ways < (int64_t)plan->num_sms * kJoinWarps) ways *= 2;
  const int64_t per = kJoinWarps / ways;
  const dim3 grid((unsigned)((n + per - 1) / per));
  if (TREE) return launch_dependent(fn, grid, kJoinThreads, 0, st, p, ways);
  fn<<<grid, kJoinThreads, 0, st>>>(p, ways);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_join(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  return launch<false>(plan, p, st);
}

cudaError_t launch_tree_join(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  return launch<true>(plan, p, st);
}

}  // namespace fp8kv
