// What the tcgen05 kernels over ragged new tokens share: bounded waits, which rows a CTA has,
// FP8 rows to swizzled fp16 operand tiles, visibility in words, packed FP32 arithmetic.
#pragma once

#include <cstdint>

#include "chunk_common.cuh"
#include "tc_ptx.cuh"

namespace fp8kv {
namespace {

using namespace tc;

constexpr int kT = kChunkTileTokens;
constexpr int kM = 128;                  // rows per tile
constexpr uint32_t kPolls = 1u << 20;    // polls per wait

template <int D>
struct RowCfg {
  static constexpr int kCh = D / 16;          // 16-byte pieces of an FP8 row
  static constexpr int kRowsIt = 32 / kCh;    // rows a warp moves at a time
  static constexpr int kIts = 32 / kRowsIt;   // times, for its 32 rows
};

// A bounded wait of a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kPolls, abort_flag));
}

// One lane of a converged warp (always the same).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Request and first packed row of a CTA.  The GPU starts CTAs in the order of their
// index, so the longest go first: requests by the positions that their rows see
// (above 32 requests, more than a warp's lanes: by their index, from the last; not
// measured against an order by length), a request's row tiles from the last, which sees
// the most, and the KV heads of a row tile side by side.  16 requests on 200 to 8000
// positions: 133 us; with requests by index and row tiles before heads, whose longest
// CTAs started last, 189.
struct TileWork {
  int b, row0;
};
__device__ __forceinline__ int tiles_of(const ChunkParams& p, int b, int rows, bool& bad) {
  if (b >= p.B) return 0;
  const ChunkRequest r = chunk_request(p, b);
  bad |= r.bad;
  return (r.n * p.G + rows - 1) / rows;
}
__device__ __forceinline__ bool locate(const ChunkParams& p, int rows, int idx, int lane, TileWork& w) {
  int total = 0;
  bool bad = false;
  if (p.B <= 32) {
    const int mine = tiles_of(p, lane, rows, bad);
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) set_status(p.status, FP8KV_STATUS_BAD_LEN);
    int key = 0, before = 0;  // tiles of the requests that go first
    if (lane < p.B) key = min(max(p.kv_len[lane], 0), p.window > 0 ? p.window : INT_MAX);
    for (int i = 0; i < p.B; ++i) {
      const int k = __shfl_sync(0xffffffffu, key, i), n = __shfl_sync(0xffffffffu, mine, i);
      if (k > key || (k == key && i > lane)) before += n;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, before <= idx && idx - before < mine);
    if (here == 0u) return false;
    const int l = __ffs(here) - 1;
    w.b = l;
    w.row0 = (__shfl_sync(0xffffffffu, before + mine, l) - 1 - idx) * rows;
    return true;
  }
  for (int b0 = 0; b0 < p.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, tiles_of(p, b0 + lane, rows, bad));
  if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) set_status(p.status, FP8KV_STATUS_BAD_LEN);
  idx = total - 1 - idx;
  if (idx < 0) return false;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int mine = tiles_of(p, b0 + lane, rows, bad);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, upto > idx);
    if (past) {
      const int l = __ffs(past) - 1;
      w.b = b0 + l;
      w.row0 = (idx - __shfl_sync(0xffffffffu, upto - mine, l)) * rows;
      return true;
    }
    idx -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// A CTA's share where every request is one row block: the partitions' length T (tiles) is the least with
// which all requests' partitions fit the `per_head` CTAs of a KV head, so that one wave of CTAs
// has nearly equal work whatever the lengths are, and no CTA's start (10 us of the weights' kernel,
// and 17 in a further wave) is paid twice on an SM.  By a whole warp; at most kShareMax requests.
// TREE: a request of up to 128 rows takes less time for a tile, so its partitions are longer by a
// quarter; one without positions has a CTA too (its rows are 0).
struct Share {
  int b, s, T, parts;  // request, partition of it, tiles of a partition, partitions of the request
  int base;            // T of a request whose partitions are not lengthened
};
constexpr int kShareRequests = kShareMax / 32;
template <bool TREE>
__device__ __forceinline__ bool share_of(const ChunkParams& p, int per_head, int idx, int lane, Share& out) {
  int t[kShareRequests], most = 1;
  bool light[kShareRequests];
#pragma unroll
  for (int i = 0; i < kShareRequests; ++i) {
    const int b = lane + 32 * i;
    t[i] = 0;
    light[i] = false;
    if (b < p.B) {
      const ChunkRequest r = chunk_request(p, b);
      if (r.bad && blockIdx.x == 0 && threadIdx.x < 32) set_status(p.status, FP8KV_STATUS_BAD_LEN);
      if (r.n > 0) {
        t[i] = (chunk_span<TREE>(p, r, 0, r.n - 1).U + kT - 1) / kT;
        if (TREE) t[i] = max(t[i], 1);
        light[i] = r.n * p.G <= kM;
      }
    }
    most = max(most, t[i]);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  int lo = 1, hi = most;  // (as many CTAs as requests: with T = most they fit)
  while (lo < hi) {
    const int T = (lo + hi) >> 1;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kShareRequests; ++i) {
      const int len = share_tiles<TREE>(T, light[i]);
      n += (t[i] + len - 1) / len;
    }
    if (__reduce_add_sync(0xffffffffu, n) <= (unsigned)per_head)
      hi = T;
    else
      lo = T + 1;
  }
  // The GPU starts CTAs in the order of their index: whole partitions first, requests' last ones,
  // which are shorter, behind them.
  out.base = lo;
  bool found = false;
#pragma unroll
  for (int rest = 0; rest < 2; ++rest)
#pragma unroll
    for (int i = 0; i < kShareRequests; ++i) {
      const int len = share_tiles<TREE>(lo, light[i]), whole = t[i] / len, parts = (t[i] + len - 1) / len;
      const int mine = rest ? parts - whole : whole;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, upto > idx && upto - mine <= idx);
      if (here && !found) {
        found = true;
        const int l = __ffs(here) - 1;
        out.b = l + 32 * i;
        out.s = __shfl_sync(0xffffffffu, (rest ? whole : 0) + idx - (upto - mine), l);
        out.T = __shfl_sync(0xffffffffu, len, l);
        out.parts = __shfl_sync(0xffffffffu, parts, l);
      }
      idx -= __shfl_sync(0xffffffffu, upto, 31);
    }
  return found;
}

// A decoder lane's 16-byte pieces of one tile (piece lane % kCh of rows it *
// kRowsIt + lane / kCh of the warp's 32).  The loads are unconditional (rows
// without a place read the pool's first one): a load under a condition is
// waited for on the spot, one after the other.  The rows' offsets come
// through shared memory: one access each, where a shuffle would take two.
template <int D>
__device__ __forceinline__ void fetch_rows(const uint8_t* base, const int64_t* place, int lane,
                                           uint4 (&w)[RowCfg<D>::kIts]) {
  using C = RowCfg<D>;
  base += (lane % C::kCh) * 16;
  place += lane / C::kCh;
#pragma unroll
  for (int it = 0; it < C::kIts; ++it) w[it] = __ldg(reinterpret_cast<const uint4*>(base + place[it * C::kRowsIt]));
}

// ... and as fp16 in the operand tile: 64-column blocks of kT rows of 128
// bytes, 16-byte chunk c of row r at c ^ (r % 8).  Odd column blocks store
// their two chunks in the other order, so that eight lanes hit eight banks.
// (ITS: of the warp's rows, as many times kRowsIt as one call stores.)
template <int D, int FMT, int ITS = RowCfg<D>::kIts>
__device__ __forceinline__ void store_rows(uint8_t* op, const uint4 (&w)[ITS], int row_base, int lane) {
  using C = RowCfg<D>;
  const int c = lane % C::kCh, db = c / 4, h0 = (c % 4) * 2;
  const bool swap = db & 1;
  const int first = swap ? h0 + 1 : h0, second = swap ? h0 : h0 + 1;
#pragma unroll
  for (int it = 0; it < ITS; ++it) {
    const int r = row_base + it * C::kRowsIt + lane / C::kCh;
    uint8_t* row = op + db * (kT * 128) + r * 128;
    uint4 a, b;
    fp8x4_to_f16<FMT>(w[it].x, a.x, a.y);
    fp8x4_to_f16<FMT>(w[it].y, a.z, a.w);
    fp8x4_to_f16<FMT>(w[it].z, b.x, b.y);
    fp8x4_to_f16<FMT>(w[it].w, b.z, b.w);
    *reinterpret_cast<uint4*>(row + ((first ^ (r & 7)) * 16)) = swap ? b : a;
    *reinterpret_cast<uint4*>(row + ((second ^ (r & 7)) * 16)) = swap ? a : b;
  }
}

// Visibility of 32 virtual tokens v0 .. v0+31 for one row, as bits.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t sees32(const ChunkRow& r, int sk, int v0) {
  return below(r.hi - v0) & (~below(r.lo - v0) | below(sk - v0));
}
// (words of the mask: nodes past the last one are bits of words that are there, or 0)
__device__ __forceinline__ uint32_t sees32(const TreeRow& r, int sk, int v0, int words) {
  const uint32_t context = below(r.hi - v0);
  uint32_t vis = context & (~below(r.lo - v0) | below(sk - v0));
  if (context != 0xFFFFFFFFu) {
    const int j0 = v0 - r.hi, w = j0 >> 5;  // node of the first token; negative: context in front
    const uint32_t lo = w >= 0 && w < words ? __ldg(r.mask + w) : 0u;
    const uint32_t hi = w + 1 >= 0 && w + 1 < words ? __ldg(r.mask + w + 1) : 0u;
    vis |= __funnelshift_r(lo, hi, j0 & 31) & ~context;
  }
  return vis;
}

// Two FP32 values in a register pair (packed arithmetic of sm_100).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace
}  // namespace fp8kv
