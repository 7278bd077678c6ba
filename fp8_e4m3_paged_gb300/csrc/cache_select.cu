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
// latency for the usual sizes: the bytes of a list are read once, eight loads of a thread in flight,
// and each of the histograms costs its CTA barriers and, in a cluster, a barrier and the peers'
// counts.  128 lists of 1000 to 40000, budget 4096: 23 us; a joint list of 131072 over 8 heads: 25 us, where
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
constexpr int kMinRun = 2048;                  // positions per CTA before a list gets a further one

template <int kThreads>
struct Shared {
  static constexpr int kWarps = kThreads / 32;
  alignas(16) uint32_t hist[kPasses][kBins];
  uint32_t tie[kWarps], above[kWarps];         // selected ones and equal ones of each warp's run
  uint32_t warp_sum[kWarps];
  uint32_t digit, left;                        // found by one thread for all
  uint32_t total[2];                           // of the CTA: above, equal
};

// Keys in the order of the weights: larger weight, larger key.  -0 is +0; a NaN is below all.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The weights of kAhead positions, kThreads apart (past the last one: that again): one head's, or the
// sums over all heads, one after another.  All loads of a head are in flight together.
template <int kThreads>
__device__ __forceinline__ void weights_at(const fp8kv_cache_select_args& a, const float* row, int i, int n,
                                           float (&x)[kAhead]) {
#pragma unroll
  for (int j = 0; j < kAhead; ++j) x[j] = __ldg(row + min(i + j * kThreads, n - 1));
  if (a.lists == 1) {
#pragma unroll 4
    for (int h = 1; h < a.num_kv_heads; ++h) {
      float y[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) y[j] = __ldg(row + h * a.score_stride_head + min(i + j * kThreads, n - 1));
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
  extern __shared__ uint32_t keys[];
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
  const bool stay = n <= kKeys;
  for (int i = tid; i < kPasses * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0u;
  __syncthreads();

  uint32_t prefix = 0u, want = (uint32_t)m;  // bits found so far; the m-th is the want-th of those with the prefix
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    uint32_t* hist = sh.hist[pass];
    const uint32_t mask = (1u << bits) - 1u;
    for (int i0 = tid; i0 < n; i0 += kAhead * kThreads) {
      uint32_t k[kAhead];
      if (pass == 0 || !stay) {
        float x[kAhead];
        weights_at<kThreads>(a, row + t0, i0, n, x);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          k[j] = key_of(x[j]);
          if (stay && i0 + j * kThreads < n) keys[i0 + j * kThreads] = k[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) k[j] = keys[min(i0 + j * kThreads, n - 1)];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j * kThreads < n && (pass == 0 || (k[j] >> (shift + bits)) == prefix))
          atomicAdd(&hist[(k[j] >> shift) & mask], 1u);
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
  const int part = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int w0 = min(warp * part, n), w1 = min(w0 + part, n);
  auto key_at = [&](int i) { return stay ? keys[i] : key_of(weight_at(a, row, t0 + i)); };
  uint32_t above = 0u, tie = 0u;
#pragma unroll 8
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key_at(i);
    above += k > cut;
    tie += k == cut;
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
#pragma unroll 4
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < w1 ? key_at(i) : 0u;
    const uint32_t up = __ballot_sync(0xffffffffu, i < w1 && k > cut), eq = __ballot_sync(0xffffffffu, i < w1 && k == cut);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t above_i = above0 + __popc(up & below), tie_i = tie0 + __popc(eq & below);
    if ((up >> lane & 1u) || ((eq >> lane & 1u) && tie_i < want))
      keep[a.sinks + above_i + min(tie_i, want)] = t0 + i;
    above0 += __popc(up);
    tie0 += __popc(eq);
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
  // CTAs per list: while the GPU has room for them (three to an SM) and each keeps kMinRun positions
  const int64_t lists = (int64_t)a.batch * a.lists;
  int ctas = 1;
  while (ctas < kClusterMax && lists * ctas * 2 <= 4 * (int64_t)sms && a.max_len / (2 * ctas) >= kMinRun) ctas *= 2;
  while (ctas < kClusterMax && (a.max_len + ctas - 1) / ctas > kKeys) ctas *= 2;
  if (lists * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // twice the threads, so twice the loads on their way, where every CTA has an SM and much to read
  const bool wide = lists * ctas <= sms && a.max_len / ctas >= 4096;
  return wide ? run<1024>(a, lists, ctas, st) : run<512>(a, lists, ctas, st);
}

}  // namespace fp8kv
