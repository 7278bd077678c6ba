// Cache move: rows of the paged cache from position first + src[k] to first + k.
//
// Bytes in, bytes out: each row that moves is read once and written once, so HBM bounds a
// large move, and a launch and the chain list -> block table -> row a small one.
//
// In place, a row's new place may be another row's old one.  Every row moves towards
// the front (src[k] >= k; others are refused), so a row k' > k has its source at k' or behind:
// new places of rows below k' never hold a source of rows from k' on.  It is
// enough, then, that rows are taken in rounds by k and that a round is written only when all rows up
// to its end have been read; later rows may be read as early as one likes.  One unit (a request's KV
// head, K and V) is walked by one CTA, or by one cluster, whose barrier in each round says that
// all CTAs' reads have arrived, and orders them before the others' writes.  (Its release waits for
// the writes of the round before it, too: 16 x 2052 rows 38.7 us, 35.4 without it, one request 9.6 and
// 8.3.  Without it, nothing but cp.async's completion would stand between one CTA's read of a row and
// another's write of it.)  To pages of their own no such order is needed.
//
// Rounds of 32 KB per CTA through shared memory: cp.async brings the rows of the next two
// rounds while this one is written, and the list and the table of the round after them are
// looked up meanwhile, so that a CTA always has rows in flight (in registers, one round at a
// time, 16 x 2052 rows of 8 heads took 58 us).  16 bytes per thread and access, eight lanes to a
// row of 128: rows are whole sectors whatever the list.
//
// 8 x 4096 rows of 8 heads (D 128, by lists, with weights) 37 us, 3.7 TB/s read and written; 16 x 2052 in place
// 39, 3.5 TB/s; a plain copy reaches 6.8.  64 accepted paths of up to five rows: 4.4 us.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "cluster.cuh"
#include "device_common.cuh"
#include "evict.h"
#include "internal.h"
#include "tc_ptx.cuh"

namespace fp8kv {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 8;                       // 16-byte pieces per thread and round
constexpr int kStages = 3;
constexpr int kStageBytes = kItems * kThreads * 16;
constexpr int kMaxPlaces = 128;                 // rows of a round (of all heads that have a list)
constexpr int kClusterMax = 8;
constexpr int kResident = 2;                    // CTAs per SM

struct Geometry {
  int rows;      // rows of a CTA's round
  int heads;     // KV heads of a CTA
  int lists;     // lists of those heads: 1 or heads
  int chunks;    // 16-byte pieces of a row of one head
  int ctas;      // CTAs of a unit: in place, of its cluster
};

struct Place {
  int64_t ks, vs, kd, vd;  // byte offsets; kd < 0: the row does not move
};

template <bool IN_PLACE>
__global__ void __launch_bounds__(kThreads, kResident) move_kernel(const __grid_constant__ fp8kv_cache_move_args a,
                                                                   const Geometry geo) {
  extern __shared__ __align__(16) uint8_t stages[];
  __shared__ Place s_place[kStages][kMaxPlaces];
  const int tid = threadIdx.x;
  const int unit = blockIdx.x / geo.ctas, rank = blockIdx.x - unit * geo.ctas;
  const int groups = a.num_kv_heads / geo.heads;
  const int b = unit / groups, g0 = (unit - b * groups) * geo.heads;
  const int asked = __ldg(a.count + b), n = min(max(asked, 0), a.max_count);
  if (asked != n && a.status && tid == 0) set_status(a.status, FP8KV_STATUS_BAD_LEN);
  const int first = a.first ? __ldg(a.first + b) : 0;
  const int32_t* from = a.block_table + b * a.block_table_stride;
  const int32_t* to = IN_PLACE ? from : a.dst_table + b * a.dst_table_stride;
  const int64_t from_end = (int64_t)a.max_blocks * a.page_size;
  const int64_t to_end = IN_PLACE ? from_end : (int64_t)a.dst_max_blocks * a.page_size;
  const int step = geo.rows * geo.ctas;
  const int n_rounds = (int)(((int64_t)n + step - 1) / step);  // (the same for all CTAs of a cluster)

  // This thread's row of a round: list l, row tid - l * rows.
  const bool finds = tid < geo.rows * geo.lists;
  const int l = tid / geo.rows, row = tid - l * geo.rows;
  const int32_t* list = a.src + b * a.src_stride_req + (a.lists > 1 ? (g0 + l) * a.src_stride_list : 0) + row;
  // Looking a round up takes three steps, one each in three successive rounds.
  int32_t s = 0, ob = 0, nb = 0;  // list entry; blocks
  int os = 0, ns = 0, k_at = 0;
  uint32_t bad = 0u;
  auto read_list = [&](int round) {  // ... of round `round`
    k_at = round * step + rank * geo.rows;
    s = -1;
    if (finds && k_at + row < n) s = __ldg(list + k_at);
  };
  auto read_table = [&]() {  // ... of the entry read
    const int k = k_at + row;
    bad = 0u;
    ob = nb = -1;
    if (!finds || k >= n) return;
    const int64_t old_pos = (int64_t)first + s, new_pos = (int64_t)first + k;
    if (s < (IN_PLACE ? k : 0)) {
      bad = FP8KV_STATUS_BAD_ENTRIES;
      return;
    }
    if (!IN_PLACE || s != k) {
      bad = FP8KV_STATUS_BAD_BLOCK;
      if (old_pos >= 0 && old_pos < from_end && new_pos >= 0 && new_pos < to_end) {
        const int op = (int)(old_pos / a.page_size), np = (int)(new_pos / a.page_size);
        os = (int)(old_pos - (int64_t)op * a.page_size);
        ns = (int)(new_pos - (int64_t)np * a.page_size);
        ob = __ldg(from + op);
        nb = __ldg(to + np);
        bad = 0u;
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
  };
  auto write_place = [&](int slot) {  // ... of the blocks read
    if (!finds) return;
    Place p = {0, 0, -1, -1};
    const int k = k_at + row;
    if (k < n && s >= (IN_PLACE ? k : 0) && (!IN_PLACE || s != k) && !(bad & FP8KV_STATUS_BAD_BLOCK)) {
      if (ob >= 0 && ob < a.num_kv_blocks && nb >= 0 && nb < a.num_kv_blocks) {
        p.ks = ob * a.kc_stride_block + os * a.kc_stride_token;
        p.vs = ob * a.vc_stride_block + os * a.vc_stride_token;
        p.kd = nb * a.kc_stride_block + ns * a.kc_stride_token;
        p.vd = nb * a.vc_stride_block + ns * a.vc_stride_token;
      } else {
        bad |= FP8KV_STATUS_BAD_BLOCK;
      }
    }
    if (bad && a.status) set_status(a.status, bad);
    s_place[slot][tid] = p;
  };

  // This thread's pieces of a round, the same in every one: the place, whether K or V, and where the
  // piece of that head's row lies in the row at offset 0.
  const int per_head = geo.rows * geo.chunks, per_cache = per_head * geo.heads;
  int piece[kItems];  // place | V << 9; -1: none
  uint8_t* base[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int x = j * kThreads + tid;
    const bool is_v = x >= per_cache;
    const int y = is_v ? x - per_cache : x, h = y / per_head, z = y - h * per_head, r = z / geo.chunks,
              c = z - r * geo.chunks;
    piece[j] = x < 2 * per_cache ? ((geo.lists > 1 ? h * geo.rows : 0) + r) | (is_v ? 512 : 0) : -1;
    base[j] = (is_v ? a.v_cache + (g0 + h) * a.vc_stride_head : a.k_cache + (g0 + h) * a.kc_stride_head) + c * 16;
  }
  auto request = [&](int round) {  // copies of a round's rows, whose places are written
    const int slot = round % kStages;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      if (piece[j] < 0) continue;
      const Place& p = s_place[slot][piece[j] & 511];
      if (p.kd >= 0)
        tc::cp_async16(stages + slot * kStageBytes + (j * kThreads + tid) * 16,
                       base[j] + (piece[j] & 512 ? p.vs : p.ks));
    }
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

  // Before the first round: rounds 0 and 1 on their way, list of round 2
#pragma unroll
  for (int r = 0; r < kStages - 1; ++r) {
    if (r < n_rounds) {
      read_list(r);
      read_table();
      write_place(r);
      __syncthreads();
      request(r);
    }
    commit();
  }
  if (kStages - 1 < n_rounds) read_list(kStages - 1);
  for (int round = 0; round < n_rounds; ++round) {
    const bool more = round + kStages - 1 < n_rounds;
    if (more) read_table();
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");  // this round's rows
    if (IN_PLACE && geo.ctas > 1)
      cluster_sync();
    else
      __syncthreads();
    const int slot = round % kStages;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      if (piece[j] < 0) continue;
      const Place& p = s_place[slot][piece[j] & 511];
      if (p.kd >= 0)
        *reinterpret_cast<uint4*>(base[j] + (piece[j] & 512 ? p.vd : p.kd)) =
            *reinterpret_cast<const uint4*>(stages + slot * kStageBytes + (j * kThreads + tid) * 16);
    }
    if (more) {
      // (its slot held the round before this one, which every thread is past)
      write_place((round + kStages - 1) % kStages);
      __syncthreads();
      request(round + kStages - 1);
      if (round + kStages < n_rounds) read_list(round + kStages);
    }
    commit();
  }
}

template <bool IN_PLACE>
cudaError_t run(const fp8kv_cache_move_args& a, const Geometry& g, int64_t grid, int rounds, cudaStream_t st) {
  static DeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(move_kernel<IN_PLACE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * kStageBytes);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = std::min(rounds, kStages) * kStageBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = g.ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = IN_PLACE && g.ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, move_kernel<IN_PLACE>, a, g);
}

}  // namespace

cudaError_t launch_cache_move(const fp8kv_cache_move_args& a, int sms, cudaStream_t st) {
  const bool in_place = a.dst_table == nullptr;
  Geometry g;
  g.chunks = (a.kv_format == FP8KV_KV_BF16 ? 2 : 1) * a.head_dim / 16;
  constexpr int cap = kItems * kThreads;
  auto rows_for = [&](int heads) {
    const int lists = a.lists > 1 ? heads : 1;
    return std::min((int)(cap / ((int64_t)2 * g.chunks * heads)), kMaxPlaces / lists);
  };
  // All heads in one CTA where their rows are a round's at most, else a unit for each.
  g.heads = rows_for(a.num_kv_heads) >= a.max_count ? a.num_kv_heads : 1;
  g.lists = a.lists > 1 ? g.heads : 1;
  g.rows = std::min(rows_for(g.heads), a.max_count);
  const int64_t units = (int64_t)a.batch * (a.num_kv_heads / g.heads);
  const int runs = (int)(((int64_t)a.max_count + g.rows - 1) / g.rows);
  // As many CTAs per unit as fill the GPU, and no more: each then has rounds to overlap.
  const int64_t slots = (int64_t)kResident * sms, want = std::max<int64_t>(1, slots / units);
  g.ctas = 1;
  if (in_place) {
    while (g.ctas < kClusterMax && 2 * g.ctas <= want && g.ctas < runs) g.ctas *= 2;
  } else {
    g.ctas = (int)std::min<int64_t>(want, runs);
    // Where that leaves the last wave less than two thirds of the others' use, four waves of shorter CTAs, of three
    // rounds at least (160 units of 2052 rows 62 -> 50 us, 320 120 -> 90; 64 units, whose waves
    // are full, 17.0 either way, and 8 units 5.9 -> 10 in shorter CTAs: those stay).  In place, where
    // a unit's CTAs wait for one another, it was no faster (51 / 51, 60 -> 66 for 224 units).
    const int64_t waves = (units * g.ctas + slots - 1) / slots;
    if (units * 2 > slots && 2 * waves * slots > 3 * units * g.ctas)
      g.ctas = (int)std::max<int64_t>(g.ctas, std::min<int64_t>((4 * slots + units - 1) / units, runs / 3));
  }
  if (units * g.ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int rounds = (int)(((int64_t)a.max_count + (int64_t)g.rows * g.ctas - 1) / ((int64_t)g.rows * g.ctas));
  return in_place ? run<true>(a, g, units * g.ctas, rounds, st) : run<false>(a, g, units * g.ctas, rounds, st);
}

}  // namespace fp8kv
