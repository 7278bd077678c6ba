// Cache selection: the positions of a request that stay in the cache, by their weights.
//
// Of a list's positions the first `sinks` and the last `recent` stay; of those between, the
// m with the largest weights, where a tie goes to the lower position.  The m-th largest
// weight is found exactly by its bits: a weight becomes a 32-bit key in the same order,
// and three histograms (11, 11 and 10 bits, from the top) fix the key of the
// m-th and how many equal ones are among the m.  A last pass writes positions in
// order, each at the number of selected ones in front of it.
//
// One thread-block cluster per list, each CTA with a run of the positions, each thread with EACH
// keys in registers, kThreads positions apart, all of whose loads are in flight together; a longer
// run is taken in pieces, which are read again (from L2) in every pass.  Bound by latency for the
// usual sizes: the bytes of a list are read once, and each of the histograms costs its CTA
// barriers and, in a cluster, a barrier and the peers' counts.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "cluster.cuh"
#include "device_common.cuh"
#include "evict.h"
#include "internal.h"

namespace fp8kv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterMax = 8;
constexpr int kBins = 2048;
constexpr int kPasses = 3;
constexpr int kMinRun = 2048;                  // positions per CTA before a list gets a further one

template <int EACH>
struct Shared {
  alignas(16) uint32_t hist[kPasses][kBins];
  uint32_t above[EACH * kWarps], tie[EACH * kWarps];  // selected ones and equal ones of a warp's 32 positions
  uint32_t warp_sum[kWarps];
  uint32_t digit, left;                        // found by one thread for all
  uint32_t total[2];                           // of the CTA: above, equal
  uint32_t run[2];                             // of the piece
};

// Keys in the order of the weights: larger weight, larger key.  -0 is +0; a NaN is below all.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Keys of EACH positions, kThreads apart (past the last one: that again): one head's weight, or
// the sum over all heads, one after another.
template <int EACH>
__device__ __forceinline__ void read_keys(const fp8kv_cache_select_args& a, const float* row, int i, int n,
                                          uint32_t (&key)[EACH]) {
  float x[EACH];
#pragma unroll
  for (int j = 0; j < EACH; ++j) x[j] = __ldg(row + min(i + j * kThreads, n - 1));
  if (a.lists == 1) {
#pragma unroll(EACH <= 8 ? 4 : 1)
    for (int h = 1; h < a.num_kv_heads; ++h) {
      float y[EACH];
#pragma unroll
      for (int j = 0; j < EACH; ++j) y[j] = __ldg(row + h * a.score_stride_head + min(i + j * kThreads, n - 1));
#pragma unroll
      for (int j = 0; j < EACH; ++j) x[j] = __fadd_rn(x[j], y[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < EACH; ++j) key[j] = key_of(x[j]);
}

// Sum of all lanes' and earlier warps' values in front of this thread's, and the CTA's total.
__device__ __forceinline__ uint32_t scan_before(uint32_t x, uint32_t* warp_sum, int lane, int warp, uint32_t& total) {
  uint32_t upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  const uint32_t mine = lane < kWarps ? warp_sum[lane] : 0u;
  total = __reduce_add_sync(0xffffffffu, mine);
  return __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0u) + upto - x;
}

template <int EACH>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ fp8kv_cache_select_args a,
                                                          const int ctas) {
  __shared__ Shared<EACH> sh;
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

  // This CTA's run of the positions between, in pieces of EACH positions per thread
  const int run = (hi - lo + ctas - 1) / ctas;
  const int t0 = (int)min((int64_t)lo + (int64_t)rank * run, (int64_t)hi), n = (int)min((int64_t)t0 + run, (int64_t)hi) - t0;
  constexpr int kPiece = EACH * kThreads;
  uint32_t key[EACH];
  auto read_piece = [&](int i0) { read_keys<EACH>(a, row + t0, i0 + tid, n, key); };
  if (n > 0) read_piece(0);
  for (int i = tid; i < kPasses * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0u;
  __syncthreads();

  uint32_t prefix = 0u, want = (uint32_t)m;  // bits found so far; the m-th is the want-th of those with the prefix
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    uint32_t* hist = sh.hist[pass];
    for (int i0 = 0; i0 < n; i0 += kPiece) {
      if (n > kPiece && (pass > 0 || i0 > 0)) read_piece(i0);
#pragma unroll
      for (int j = 0; j < EACH; ++j)
        if (i0 + tid + j * kThreads < n && (pass == 0 || (key[j] >> (shift + bits)) == prefix))
          atomicAdd(&hist[(key[j] >> shift) & ((1u << bits) - 1u)], 1u);
    }
    if (ctas > 1)
      cluster_sync();
    else
      __syncthreads();
    // bins from the top: thread tid holds four, from kBins - 1 - 4 tid down
    constexpr int kEach = kBins / kThreads;
    uint32_t c[kEach], sum = 0u;
#pragma unroll
    for (int j = 0; j < kEach; ++j) c[j] = 0u;
    for (int q = 0; q < ctas; ++q) {
      const uint4 x = ctas == 1 ? *reinterpret_cast<const uint4*>(hist + kBins - 4 - 4 * tid)
                                : peer_load4(hist + kBins - 4 - 4 * tid, q);
      c[0] += x.w;
      c[1] += x.z;
      c[2] += x.y;
      c[3] += x.x;
    }
    static_assert(kEach == 4, "a thread's bins are one load");
#pragma unroll
    for (int j = 0; j < kEach; ++j) sum += c[j];
    uint32_t total;
    uint32_t before = scan_before(sum, sh.warp_sum, lane, warp, total);
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
  uint32_t above0 = 0u, tie0 = 0u;  // in front of this CTA's run
  if (ctas > 1) {
    uint32_t above = 0u, tie = 0u;
    for (int i0 = 0; i0 < n; i0 += kPiece) {
      if (n > kPiece) read_piece(i0);
#pragma unroll
      for (int j = 0; j < EACH; ++j)
        if (i0 + tid + j * kThreads < n) {
          above += key[j] > cut;
          tie += key[j] == cut;
        }
    }
    if (tid < 2) sh.total[tid] = 0u;
    __syncthreads();
    above = __reduce_add_sync(0xffffffffu, above);
    tie = __reduce_add_sync(0xffffffffu, tie);
    if (lane == 0) {
      atomicAdd(&sh.total[0], above);
      atomicAdd(&sh.total[1], tie);
    }
    cluster_sync();
    for (int q = 0; q < rank; ++q) {
      above0 += peer_load(&sh.total[0], q);
      tie0 += peer_load(&sh.total[1], q);
    }
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = 0; i0 < n; i0 += kPiece) {
    if (n > kPiece) read_piece(i0);
    // counts of each 32 positions, in order, then what lies in front of them
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const bool in = i0 + tid + j * kThreads < n;
      const uint32_t up = __ballot_sync(0xffffffffu, in && key[j] > cut), eq = __ballot_sync(0xffffffffu, in && key[j] == cut);
      if (lane == 0) {
        sh.above[j * kWarps + warp] = __popc(up);
        sh.tie[j * kWarps + warp] = __popc(eq);
      }
    }
    __syncthreads();
    constexpr int kCounts = EACH * kWarps, kPer = (kCounts + kThreads - 1) / kThreads;
    // above in the low half, ties in the high one: a piece has at most 2^15 of both
    static_assert(kPiece < 65536, "16 bits");
    uint32_t x[kPer], sum = 0u;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      x[j] = i < kCounts ? sh.above[i] | sh.tie[i] << 16 : 0u;
      sum += x[j];
    }
    uint32_t total;
    uint32_t before = scan_before(sum, sh.warp_sum, lane, warp, total);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      if (i < kCounts) {
        sh.above[i] = before & 0xFFFFu;
        sh.tie[i] = before >> 16;
      }
      before += x[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int i = i0 + tid + j * kThreads;
      const bool up = i < n && key[j] > cut, eq = i < n && key[j] == cut;
      const uint32_t ups = __ballot_sync(0xffffffffu, up), eqs = __ballot_sync(0xffffffffu, eq);
      const uint32_t above_i = above0 + sh.above[j * kWarps + warp] + __popc(ups & below);
      const uint32_t tie_i = tie0 + sh.tie[j * kWarps + warp] + __popc(eqs & below);
      if (up || (eq && tie_i < want)) keep[a.sinks + above_i + min(tie_i, want)] = t0 + i;
    }
    above0 += total & 0xFFFFu;
    tie0 += total >> 16;
    __syncthreads();  // the next piece's counts
  }
  if (ctas > 1) cluster_sync();  // peers may still read this CTA's counts
}

template <int EACH>
cudaError_t run(const fp8kv_cache_select_args& a, int64_t lists, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(lists * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, select_kernel<EACH>, a, ctas);
}

}  // namespace

cudaError_t launch_cache_select(const fp8kv_cache_select_args& a, int sms, cudaStream_t st) {
  // CTAs per list: while the GPU has room for them (four to an SM) and each keeps kMinRun positions
  const int64_t lists = (int64_t)a.batch * a.lists;
  int ctas = 1;
  while (ctas < kClusterMax && lists * ctas * 2 <= 4 * (int64_t)sms && a.max_len / (2 * ctas) >= kMinRun) ctas *= 2;
  if (lists * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int run_len = (a.max_len + ctas - 1) / ctas;
  if (run_len <= 4 * kThreads) return run<4>(a, lists, ctas, st);
  if (run_len <= 12 * kThreads) return run<12>(a, lists, ctas, st);
  return run<32>(a, lists, ctas, st);
}

}  // namespace fp8kv
