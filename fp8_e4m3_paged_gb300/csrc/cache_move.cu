// Cache move: rows of the paged cache from position first + src[k] to first + k.
//
// Bytes in, bytes out: each row that moves is read once and written once, so HBM bounds a
// large move, and a launch and the chain list -> block table -> row a small one.
//
// In place, a row's new place may be another row's old one.  Every row moves towards
// the front (src[k] >= k; others are refused), so a row k' > k has its source at k' or behind:
// new places of rows below k' never hold a source of rows from k' on.  It is
// enough, then, that rows are taken in runs by k and that a run is written only when all rows up to
// its end have been read.  One unit (a request's KV head, K and V) is therefore walked
// by one CTA, or by one cluster in rounds: each CTA reads its share of the round into registers,
// the cluster's barrier says that all have, and the shares are written.  The barrier's
// release and acquire order the reads before the writes.  To pages of their own no such order is
// needed, and every run has a CTA.
// 16 bytes per thread and access, eight lanes to a row of 128: rows are whole
// sectors whatever the list.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "cluster.cuh"
#include "device_common.cuh"
#include "evict.h"

namespace fp8kv {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 8;                       // 16-byte pieces per thread and round
constexpr int kMaxPlaces = 256;                 // rows of a round (of all heads that have a list)
constexpr int kClusterMax = 8;

struct Geometry {
  int rows;      // rows of a CTA's round
  int heads;     // KV heads of a CTA
  int lists;     // lists of those heads: 1 or heads
  int chunks;    // 16-byte pieces of a row of one head
  int ctas;      // in place: CTAs of a cluster; else runs of a unit
};

struct Place {
  int64_t ks, vs, kd, vd;  // byte offsets; kd < 0: the row does not move
};

template <bool IN_PLACE>
__global__ void __launch_bounds__(kThreads) move_kernel(const __grid_constant__ fp8kv_cache_move_args a,
                                                        const Geometry geo) {
  __shared__ Place s_place[kMaxPlaces];
  const int tid = threadIdx.x;
  const int rank = blockIdx.x % geo.ctas;
  const int unit = blockIdx.x / geo.ctas;
  const int groups = a.num_kv_heads / geo.heads;
  const int b = unit / groups, g0 = (unit - b * groups) * geo.heads;
  const int asked = __ldg(a.count + b), n = min(max(asked, 0), a.max_count);
  if (asked != n && a.status && tid == 0) set_status(a.status, FP8KV_STATUS_BAD_LEN);
  const int first = a.first ? __ldg(a.first + b) : 0;
  const int32_t* src0 = a.src + b * a.src_stride_req + (a.lists > 1 ? g0 * a.src_stride_list : 0);
  const int32_t* from = a.block_table + b * a.block_table_stride;
  const int32_t* to = IN_PLACE ? from : a.dst_table + b * a.dst_table_stride;
  const int64_t from_end = (int64_t)a.max_blocks * a.page_size;
  const int64_t to_end = IN_PLACE ? from_end : (int64_t)a.dst_max_blocks * a.page_size;
  const int step = geo.rows * geo.ctas;
  const int n_rounds = IN_PLACE ? (n + step - 1) / step : 1;
  const int per_head = geo.rows * geo.chunks, per_cache = per_head * geo.heads;
  for (int round = 0; round < n_rounds; ++round) {
    const int k0 = round * step + rank * geo.rows;
    if (!IN_PLACE && k0 >= n) return;
    // ------------------------------------------------ places of the round's rows
    for (int x = tid; x < geo.rows * geo.lists; x += kThreads) {
      const int l = x / geo.rows, k = k0 + x - l * geo.rows;
      Place p = {0, 0, -1, -1};
      if (k < n) {
        const int32_t s = __ldg(src0 + l * a.src_stride_list + k);
        const int64_t old_pos = (int64_t)first + s, new_pos = (int64_t)first + k;
        uint32_t bad = 0u;
        if (s < (IN_PLACE ? k : 0)) {
          bad = FP8KV_STATUS_BAD_ENTRIES;
        } else {
          if (!IN_PLACE || s != k) {
            bad = FP8KV_STATUS_BAD_BLOCK;
            if (old_pos >= 0 && old_pos < from_end && new_pos >= 0 && new_pos < to_end) {
              const int op = (int)(old_pos / a.page_size), np = (int)(new_pos / a.page_size);
              const int os = (int)(old_pos - (int64_t)op * a.page_size), ns = (int)(new_pos - (int64_t)np * a.page_size);
              const int64_t ob = __ldg(from + op), nb = __ldg(to + np);
              if (ob >= 0 && ob < a.num_kv_blocks && nb >= 0 && nb < a.num_kv_blocks) {
                bad = 0u;
                p.ks = ob * a.kc_stride_block + os * a.kc_stride_token;
                p.vs = ob * a.vc_stride_block + os * a.vc_stride_token;
                p.kd = nb * a.kc_stride_block + ns * a.kc_stride_token;
                p.vd = nb * a.vc_stride_block + ns * a.vc_stride_token;
              }
            }
          }
          if (a.score) {
            // weights of the list's heads
            const int h0 = a.lists > 1 ? g0 + l : g0, h1 = a.lists > 1 ? h0 + 1 : g0 + geo.heads;
            if (old_pos >= 0 && old_pos < a.max_len && new_pos >= 0 && new_pos < a.max_len) {
              for (int h = h0; h < h1; ++h)
                a.score_out[b * a.score_out_stride_req + h * a.score_out_stride_head + new_pos] =
                    __ldg(a.score + b * a.score_stride_req + h * a.score_stride_head + old_pos);
            } else {
              bad |= FP8KV_STATUS_BAD_LEN;
            }
          }
        }
        if (bad && a.status) set_status(a.status, bad);
      }
      s_place[x] = p;
    }
    __syncthreads();
    // ------------------------------------------------ read, wait for all readers, write
    // (rows that do not move read the pool's first row: loads without conditions)
    uint4 w[kItems];
    uint8_t* dst[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int x = j * kThreads + tid;
      const bool is_v = x >= per_cache;
      const int y = is_v ? x - per_cache : x, h = y / per_head, z = y - h * per_head, r = z / geo.chunks,
                c = z - r * geo.chunks;
      dst[j] = nullptr;
      w[j] = make_uint4(0, 0, 0, 0);
      if (x < 2 * per_cache) {
        const Place& p = s_place[(geo.lists > 1 ? h * geo.rows : 0) + r];
        uint8_t* base = is_v ? a.v_cache + (g0 + h) * a.vc_stride_head : a.k_cache + (g0 + h) * a.kc_stride_head;
        w[j] = __ldcg(reinterpret_cast<const uint4*>(base + (is_v ? p.vs : p.ks) + c * 16));
        if (p.kd >= 0) dst[j] = base + (is_v ? p.vd : p.kd) + c * 16;
      }
    }
    if (IN_PLACE) {
      if (geo.ctas > 1)
        cluster_sync();
      else
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j)
      if (dst[j]) *reinterpret_cast<uint4*>(dst[j]) = w[j];
    __syncthreads();  // the next round's places
  }
}

}  // namespace

cudaError_t launch_cache_move(const fp8kv_cache_move_args& a, cudaStream_t st) {
  const bool in_place = a.dst_table == nullptr;
  Geometry g;
  g.chunks = (a.kv_format == FP8KV_KV_BF16 ? 2 : 1) * a.head_dim / 16;
  constexpr int cap = kItems * kThreads;
  auto rows_for = [&](int heads) {
    const int lists = a.lists > 1 ? heads : 1;
    return std::min(cap / (2 * g.chunks * heads), kMaxPlaces / lists);
  };
  // All heads in one CTA where their rows are a round's at most, else a unit for each.
  g.heads = rows_for(a.num_kv_heads) >= a.max_count ? a.num_kv_heads : 1;
  g.lists = a.lists > 1 ? g.heads : 1;
  g.rows = std::min(rows_for(g.heads), a.max_count);
  const int runs = (int)(((int64_t)a.max_count + g.rows - 1) / g.rows);
  g.ctas = in_place ? 1 : runs;
  if (in_place)
    while (g.ctas < kClusterMax && g.ctas < runs) g.ctas *= 2;
  const int64_t grid = (int64_t)a.batch * (a.num_kv_heads / g.heads) * g.ctas;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = g.ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = in_place && g.ctas > 1 ? 1 : 0;
  return in_place ? cudaLaunchKernelEx(&cfg, move_kernel<true>, a, g) : cudaLaunchKernelEx(&cfg, move_kernel<false>, a, g);
}

}  // namespace fp8kv
