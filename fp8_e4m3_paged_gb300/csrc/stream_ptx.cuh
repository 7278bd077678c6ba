// What the streaming kernels (mma.sync, cp.async rings per warp) share.
#pragma once

#include <cstdint>

#include "chunk_common.cuh"

namespace fp8kv {
namespace {

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t word(const uint4& w, int i) {
  return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// The request with the r-th most positions (at most THREADS requests, the CTA's threads); `key` is room
// for THREADS + 1 (a static array would cost the fourth CTA of an SM).
template <int THREADS>
__device__ __forceinline__ int by_length(const ChunkParams& p, int* key, int r) {
  const int t = threadIdx.x;
  int mine = -1;
  if (t < p.B) {
    const ChunkRequest q = chunk_request(p, t);
    if (q.n > 0) mine = p.window > 0 ? min(q.kv, (int)min((int64_t)p.window + p.sinks, (int64_t)INT_MAX)) : q.kv;
    key[t] = mine;
  }
  __syncthreads();
  if (t < p.B) {
    int rank = 0;
    for (int i = 0; i < p.B; ++i) {
      const int k = key[i];
      rank += k > mine || (k == mine && i < t);
    }
    if (rank == r) key[THREADS] = t;
  }
  __syncthreads();
  const int b = key[THREADS];
  __syncthreads();
  return b;
}

}  // namespace
}  // namespace fp8kv
