// Cache selection: the positions of a request that stay in the cache, by their weights.
//
// Of a list's positions the first `sinks` and the last `recent` stay; of those between, the
// m with the largest weights, where a tie goes to the lower position.  The m-th largest
// weight is found exactly by its bits: a weight becomes a 32-bit key in the same order,
// and three histograms (11, 11 and 10 bits, from the top) fix the key of the
// m-th and how many equal ones are among the m.  A last pass writes positions in
// order, each at the number of selected ones in front of it.
//
// One thread-block cluster per list, each CTA with a run of the positions, whose keys stay in
// shared memory after the first read (up to kKeys; longer runs are read again, from L2).  Bound by
// latency and by instructions per key: the bytes of a list are read once, eight loads of a thread in
// flight, and keys leave shared memory in fours (one at a time, with tests for the end of the run on
// each: 25.4 us instead of 20.8 for the first case below); each of the histograms costs its CTA
// barriers and, in a cluster, a barrier and the peers' counts (two CTAs 1.3 us, four 3, eight 7).
// 128 lists of 1000 to 40000, budget 4096: 20.8 us; a joint list of 131072 over 8 heads: 23.6, where
// eight SMs read 4 MB.  (Keys in registers, all loops unrolled: twice the time, most of it fetching instructions.)
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "cluster.cuh"
#include "device_common.cuh"
#include "evict.h"
#include "internal.h"

namespace fp8kv {
namespace {

constexpr int kClusterMax = 8;
constexpr int kBins = 2048;
constexpr int kPasses = 3;
constexpr int kAhead = 8;                      // positions of a thread whose loads are in flight together
constexpr int kKeys = 49152;                   // keys of a CTA's run that stay in shared memory
constexpr int kMinRun = 4096;                  // positions per CTA before a list gets a further one

template <int kThreads>
struct Shared {
  static constexpr int kWarps = kThreads / 32;
  alignas(16) uint32_t hist[kPasses][kBins];
  uint32_t tie[kWarps], above[kWarps];         // of each warp's run: keys equal to the cut, and above it
  uint32_t warp_sum[kWarps];
  uint32_t digit, left;                        // found by one thread for all
  uint32_t total[2];                           // of the CTA: above, equal
};

// Keys in the order of the weights: larger weight, larger key.  -0 is +0; a NaN is below all.  0 is no
// position's key: places behind the last one hold it, are below the cut whatever it is, and need no test.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return x != x ? 1u : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// The weights of kAhead positions, kThreads apart, from `row` on (FULL; else of those below n, past them the last
// one again): one head's, or the sums over all heads, one after another.  All loads of a head are in flight together.
template <int kThreads, bool FULL>
__device__ __forceinline__ void weights_at(const fp8kv_cache_select_args& a, const float* row, int n, float (&x)[kAhead]) {
#pragma unroll
  for (int j = 0; j < kAhead; ++j) x[j] = __ldg(row + (FULL ? j * kThreads : min(j * kThreads, n - 1)));
  if (a.lists == 1) {
#pragma unroll 4
    for (int h = 1; h < a.num_kv_heads; ++h) {
      row += a.score_stride_head;
      float y[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) y[j] = __ldg(row + (FULL ? j * kThreads : min(j * kThreads, n - 1)));
#pragma unroll
      for (int j = 0; j < kAhead; ++j) x[j] = __fadd_rn(x[j], y[j]);
    }
  }
}
__device__ __forceinline__ float weight_at(const fp8kv_cache_select_args& a, const float* row, int t) {
  float x = __ldg(row + t);
  if (a.lists == 1)
    for (int h = 1; h < a.num_kv_heads; ++h) x = __fadd_rn(x, __ldg(row + h * a.score_stride_head + t));
  return x;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 3 : 1) select_kernel(const __grid_constant__ fp8kv_cache_select_args a,
                                                             const int ctas) {
  extern __shared__ __align__(16) uint32_t keys[];
  constexpr int kWarps = kThreads / 32;
  __shared__ Shared<kThreads> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = ctas > 1 ? cluster_rank() : 0;
  const int unit = blockIdx.x / ctas, b = unit / a.lists, l = unit - b * a.lists;
  const float* row = a.score + b * a.score_stride_req + l * a.score_stride_head;
  int32_t* keep = a.keep + b * a.keep_stride_req + l * a.keep_stride_list;
  const int asked = __ldg(a.kv_len + b), len = min(max(asked, 0), a.max_len);
  if (asked != len && a.status && tid == 0 && rank == 0) set_status(a.status, FP8KV_STATUS_BAD_LEN);
  const int kept = min(len, a.budget);
  if (l == 0 && rank == 0 && tid == 0) a.n_keep[b] = kept;
  if (len <= a.budget) {
    for (int t = rank * kThreads + tid; t < len; t += ctas * kThreads) keep[t] = t;
    return;  // (every CTA of the cluster)
  }
  const int lo = a.sinks, hi = len - a.recent, m = a.budget - a.sinks - a.recent;  // sinks + recent <= budget < len
  for (int t = rank * kThreads + tid; t < a.sinks; t += ctas * kThreads) keep[t] = t;
  for (int t = rank * kThreads + tid; t < a.recent; t += ctas * kThreads) keep[a.sinks + m + t] = hi + t;
  if (m == 0) return;

  // This CTA's run of the positions between, and each warp's part of it (whole 32s)
  const int run = ((hi - lo + ctas - 1) / ctas + 31) / 32 * 32;
  const int t0 = min(lo + rank * run, hi), n = min(t0 + run, hi) - t0;
  const int n4 = (n + 3) / 4 * 4;  // ... with the places behind the last position, so that keys are read in fours
  const bool stay = n4 <= kKeys;
  auto keys_at = [&](int i) {  // of positions i .. i + 3 of the run
    if (stay) return *reinterpret_cast<const uint4*>(keys + i);
    uint32_t k[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = i + j < n ? key_of(weight_at(a, row, t0 + i + j)) : 0u;
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  for (int i = tid; i < kPasses * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0u;
  __syncthreads();

  uint32_t prefix = 0u, want = (uint32_t)m;  // bits found so far; the m-th is the want-th of those with the prefix
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    uint32_t* hist = sh.hist[pass];
    if (pass == 0) {
      for (int i0 = tid; i0 < n4; i0 += kAhead * kThreads) {
        float x[kAhead];
        if (i0 - tid + kAhead * kThreads <= n) {
          weights_at<kThreads, true>(a, row + t0 + i0, n, x);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const uint32_t k = key_of(x[j]);
            if (stay) keys[i0 + j * kThreads] = k;
            atomicAdd(&hist[k >> shift], 1u);
          }
        } else {
          const int i = min(i0, n - 1);
          weights_at<kThreads, false>(a, row + t0 + i, n - i, x);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const int at = i0 + j * kThreads;
            const uint32_t k = at < n ? key_of(x[j]) : 0u;
            if (stay && at < n4) keys[at] = k;
            if (at < n) atomicAdd(&hist[k >> shift], 1u);
          }
        }
      }
    } else {
      const uint32_t base = prefix << (shift + bits), range = 1u << (shift + bits);
#pragma unroll 2
      for (int i = 4 * tid; i < n; i += 4 * kThreads) {
        const uint4 k4 = keys_at(i);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k[j] - base < range) atomicAdd(&hist[(k[j] - base) >> shift], 1u);
      }
    }
    if (ctas > 1)
      cluster_sync();
    else
      __syncthreads();
    // bins from the top: a thread holds four, from kBins - 1 - 4 tid down
    constexpr int kEach = 4;
    static_assert(kBins <= kEach * kThreads, "a thread's bins are one load");
    uint32_t c[kEach] = {0u, 0u, 0u, 0u};
    if (kEach * tid < kBins) {
#pragma unroll 4
      for (int q = 0; q < ctas; ++q) {
        const uint4 x = ctas == 1 ? *reinterpret_cast<const uint4*>(hist + kBins - kEach - kEach * tid)
                                  : peer_load4(hist + kBins - kEach - kEach * tid, q);
        c[0] += x.w;
        c[1] += x.z;
        c[2] += x.y;
        c[3] += x.x;
      }
    }
    const uint32_t sum = c[0] + c[1] + c[2] + c[3];
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0u) + upto - sum;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (before < want && want <= before + c[j]) {  // exactly one bin of all
        sh.digit = (uint32_t)(kBins - 1 - 4 * tid - j);
        sh.left = want - before;
      }
      before += c[j];
    }
    __syncthreads();
    prefix = (prefix << bits) | sh.digit;
    want = sh.left;
  }
  const uint32_t cut = prefix;  // keys above it stay, and the first `want` equal ones

  // ------------------------------------------------ positions in order
  constexpr int kSpan = 128;  // of a warp at a time: four of each lane
  const int part = ((n + kWarps - 1) / kWarps + kSpan - 1) / kSpan * kSpan;
  const int w0 = min(warp * part, n), w1 = min(w0 + part, n);
  uint32_t above = 0u, tie = 0u;
#pragma unroll 2
  for (int i = w0 + 4 * lane; i < w1; i += kSpan) {
    const uint4 k4 = keys_at(i);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      above += k[j] > cut;
      tie += k[j] == cut;
    }
  }
  above = __reduce_add_sync(0xffffffffu, above);
  tie = __reduce_add_sync(0xffffffffu, tie);
  if (lane == 0) {
    sh.above[warp] = above;
    sh.tie[warp] = tie;
  }
  __syncthreads();
  uint32_t above0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.above[lane] : 0u);
  uint32_t tie0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.tie[lane] : 0u);
  if (ctas > 1) {
    if (tid == kThreads - 1) {
      sh.total[0] = above0 + above;
      sh.total[1] = tie0 + tie;
    }
    cluster_sync();
    for (int q = 0; q < rank; ++q) {
      above0 += peer_load(&sh.total[0], q);
      tie0 += peer_load(&sh.total[1], q);
    }
  }
#pragma unroll 2
  for (int i0 = w0; i0 < w1; i0 += kSpan) {
    const int i = i0 + 4 * lane;
    const uint4 k4 = i < w1 ? keys_at(i) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    uint32_t mine = 0u;  // above it, and equal ones << 16
#pragma unroll
    for (int j = 0; j < 4; ++j) mine += k[j] > cut ? 1u : k[j] == cut ? 0x10000u : 0u;
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
    uint32_t above_i = above0 + ((upto - mine) & 0xFFFFu), tie_i = tie0 + ((upto - mine) >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool up = k[j] > cut, eq = k[j] == cut;
      if (up || (eq && tie_i < want)) keep[a.sinks + above_i + min(tie_i, want)] = t0 + i + j;
      above_i += up;
      tie_i += eq;
    }
    above0 += all & 0xFFFFu;
    tie0 += all >> 16;
  }
  if (ctas > 1) cluster_sync();  // peers may still read this CTA's counts
}

template <int kThreads>
cudaError_t run(const fp8kv_cache_select_args& a, int64_t lists, int ctas, cudaStream_t st) {
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(select_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeys * 4);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(lists * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 4 * std::min(kKeys, ((a.max_len + ctas - 1) / ctas + 31) / 32 * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, select_kernel<kThreads>, a, ctas);
}

}  // namespace

cudaError_t launch_cache_select(const fp8kv_cache_select_args& a, int sms, cudaStream_t st) {
  // CTAs per list: while every CTA has an SM and keeps kMinRun positions.  (More CTAs than that start late,
  // since a cluster waits until all of its CTAs have room side by side: 64 lists of 20000 in clusters of two 13 us, in
  // clusters of eight on 512 threads, four times as many CTAs as SMs, 53.  16 lists of 32000: four CTAs 13.2,
  // eight 21.)
  const int64_t lists = (int64_t)a.batch * a.lists;
  int ctas = 1;
  while (ctas < kClusterMax && lists * ctas * 2 <= sms && a.max_len / (2 * ctas) >= kMinRun) ctas *= 2;
  while (ctas < kClusterMax && (a.max_len + ctas - 1) / ctas > kKeys) ctas *= 2;
  if (lists * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // Twice the threads, so twice the loads on their way, where every CTA has an SM, or its keys leave no room for
  // another one, and much to read (128 lists of up to 40000: 25 / 33 us before keys were read in fours).
  const bool wide = (lists * ctas <= sms || a.max_len / ctas > 22000) && a.max_len / ctas >= 4096;
  return wide ? run<1024>(a, lists, ctas, st) : run<512>(a, lists, ctas, st);
}

}  // namespace fp8kv
