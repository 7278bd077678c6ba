// Gathered weights for many query vectors: two passes of tcgen05 products over K.
//
//   rows     S = Q . K^T (M = 128 query vectors, N = 128 positions): a thread has a row, and leaves
//            its maximum and sum, M_r and L_r, per partition of the positions;
//   columns  S = K . Q^T (M = 128 positions, N = 128 query vectors): a thread has a position,
//            and adds up 2^(S_tr c_r - M_r) / L_r over the rows that see it.
//
// Every product is computed twice (the column sums need all of M and L first); kept
// logits, as the streaming kernel has them, would be 4 bytes per product: more than K from the second
// row of a group on.  Both orientations take the same swizzled operand tiles, with the roles
// exchanged, so the two passes are one kernel; a position's sum stays within a thread, in
// a fixed order, without atomics.
//
// Twenty-four warps: four groups of four, each with one S buffer (128 columns; the four are all of
// TMEM), whose first warp issues the group's next product as soon as the last one is read; two teams of four decode K,
// FP8 rows brought by cp.async into a ring of tiles, to fp16.  While one group waits for its product,
// the others have 32 columns at a time in registers: four warps on each scheduler, where two
// groups with two buffers each, ahead of the tensor core, took 2500 cycles for 128 x 128, most of it
// latencies of one warp's instructions.  With two row tiles two groups share each, K tile after
// K tile; with one, the groups take every fourth K tile.
// The column pass walks several row blocks with the same positions (their sums in shared
// memory), so that a prompt of n tokens leaves n / col_part x groups partial sums and not n^2 / 128.
//
// No unit is full: of a tile of 256 x 128 in the row pass (2800 cycles) exponentials take 1024, products 1088,
// and 1750 are issue slots; the rest are hand-offs between the groups, the tensor core and the decoders.
// Prompt of 8192 tokens, 32 heads over 8, D 128: 820 us for both passes (335 rows, 480 columns; 2.7e11
// operations each, 0.67 PFLOP/s).  Last 32 rows of four prompts of 8000 to 60000: 128 us (0.95 TB/s of K, twice).
//
// Every wait is bounded, as in the attention's tile kernel.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "score_common.cuh"
#include "tile_rows.cuh"

namespace fp8kv {
namespace {

constexpr int kGroups = 4;
constexpr int kEpilogue = kGroups * 128;         // threads
constexpr int kTeams = 2;                        // of four decoder warps: every other K tile each
constexpr int kThreadsT = kEpilogue + kTeams * 128;
constexpr int kMetaHead = 12288;
constexpr int kCols = 32;                        // columns in registers
// Maxima (base 2) from which on both passes round a logit before the maximum is taken off, and the column pass keeps 1 / l
// apart.  Below, m + log2 l is one FP32 number below 2^7 (l < 2^66), which moves all of a row's weights by at most 2^-18 ln 2 =
// 2.6e-6, and a row's logits are rounded in one pass at the most, 2^-18 again.  (At 2^22, from which on it is a
// matter of finite results alone, a row's weights summed to 1 within 2^-24 m ln 2 only: 4e-5 at 2^10, 9 % below 2^22.)
// Past it the prompt of 8192 tokens takes 1.10 ms, the last rows 157 us.
constexpr float kFar = 64.f;

template <int D>
struct Cfg : RowCfg<D> {
  static constexpr int kNQ = D == 256 ? 1 : 2;                      // row tiles
  static constexpr int kRows = kNQ * kM;
  static constexpr int kStages = D == 256 ? 1 : 2;                   // K tiles, as fp16
  static constexpr int kRing = D == 256 ? 1 : D == 128 ? 2 : 4;      // ... on their way, as bytes, of each team
  static constexpr int kOpBytes = kT * D * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kNQ * kOpBytes;
  static constexpr int kRawBytes = kT * D;
  static constexpr int kOffRaw = kOffK + kStages * kOpBytes;
  static constexpr int kOffMeta = kOffRaw + kTeams * kRing * kRawBytes;
  static constexpr int kMetaBytes = kMetaHead + 2 * kScoreAccTokens * 4;
  // (at least half an SM's shared memory: one CTA per SM, which takes all of its TMEM)
  static constexpr int kSmem = (kOffMeta + kMetaBytes > 118000 ? kOffMeta + kMetaBytes : 118000) + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Meta {
  uint64_t k_full[4], k_empty[2];     // per tile (% 4, % 2)
  uint64_t s_full[kGroups], s_empty[kGroups], drain[kGroups];
  alignas(16) uint32_t valid[8][4];   // per tile (% 8): positions whose block is in range
  int64_t place[4 * kTeams][32];      // per decoder warp: byte offsets of its rows
  alignas(16) float c[256], ml[256];           // rows: logit factor; -(maximum + log2 of the sum)
  alignas(16) float m[256], inv[256];          // ... apart: -maximum; 1 / sum
  alignas(16) int hi[256];            // rows: positions below are seen (0: a row that is not there)
  float back[256];
  float2 other[kGroups - 1][128];     // rows: (maximum, sum) of the other groups with the same rows
  uint32_t tmem, abort;
};
static_assert(sizeof(Meta) <= kMetaHead, "meta block");

// The K tiles of a CTA: row blocks [r0, r1), of each the positions from u0 on that its rows see, up to u1.
struct Walk {
  int u0, u1, r0, r1;
  int base, G, rows, n;  // first new token's position, group, rows of a block, new tokens
  __device__ __forceinline__ int last_of(int rb) const {  // positions that the block's last row sees
    return base + (min((rb + 1) * rows, n * G) - 1) / G + 1;
  }
  __device__ __forceinline__ int tiles_of(int rb) const { return (min(u1, last_of(rb)) - u0 + kT - 1) / kT; }
};

// Decoders: every other K tile of the walk, in order.  A tile costs its warps some 250 instructions in
// a chain (the copies' completion, the stage, the conversions, the next copies and block ids), one
// warp to a scheduler: two teams, so that a tile is ready twice as often.
template <int D, int FMT, bool COLS>
__device__ __forceinline__ bool decode_k(const ChunkParams& p, Meta& mt, uint8_t* smem, int b, int g, const Walk& walk,
                                         int team, int w, int lane) {
  using C = Cfg<D>;
  constexpr int NS = C::kStages, R = C::kRing;
  volatile uint32_t* const abort_flag = &mt.abort;
  const uint8_t* kbase = p.k_cache + g * p.ksh + (lane % C::kCh) * 16;
  const int32_t* table = p.block_table + (int64_t)b * p.bt_stride;
  int64_t* place = mt.place[4 * team + w];
  // a lane copies, and reads back, piece lane % kCh of rows it * kRowsIt + lane / kCh of the warp's 32
  uint8_t* raw = smem + C::kOffRaw + team * R * C::kRawBytes + (32 * w + lane / C::kCh) * D + (lane % C::kCh) * 16;
  int rb = walk.r0, j = 0, n_tiles = walk.tiles_of(rb);  // the next tile to ask for: row block, tile of it
  auto forward = [&]() {
    if (rb < walk.r1 && ++j == n_tiles) {
      j = 0;
      if (++rb < walk.r1) n_tiles = walk.tiles_of(rb);
    }
  };
  struct Ask {
    int blk, slot;
    bool in;
  };
  auto ask = [&]() {
    Ask a = {-1, 0, false};
    if (rb >= walk.r1) return a;
    const int v = walk.u0 + j * kT + 32 * w + lane;
    const int page = div_page(v, p.page_size, p.page_div);
    a.slot = v - page * p.page_size;
    a.in = v < walk.u1;
    if (a.in) a.blk = __ldg(table + page);
    for (int i = 0; i < kTeams; ++i) forward();
    return a;
  };
  auto request = [&](const Ask& a, int slot) {  // returns the rows that are there
    const bool ok = a.blk >= 0 && a.blk < p.num_kv_blocks;
    if (a.in && !ok) set_status(p.status, FP8KV_STATUS_BAD_BLOCK);
    const uint32_t rows = __ballot_sync(0xffffffffu, ok);
    if (rows == 0u) return rows;  // (their logits are masked, whatever the bytes)
    place[lane] = ok ? a.blk * p.ksb + (int64_t)a.slot * p.kst : 0;
    __syncwarp();
    // Rows that are not there are not read: one row in their place, the same for every CTA, took 5 us
    // of each CTA's 15 in waiting for its part of the L2.
#pragma unroll
    for (int it = 0; it < C::kIts; ++it) {
      const int r = it * C::kRowsIt + lane / C::kCh;
      cp_async16_or_zero(raw + slot * C::kRawBytes + it * C::kRowsIt * D, kbase + place[r], (rows >> r) & 1u ? 16u : 0u);
    }
    __syncwarp();
    return rows;
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
  for (int i = 0; i < team; ++i) forward();
  uint32_t there[R];
  Ask next;
  {
    Ask first[R + 1];
#pragma unroll
    for (int i = 0; i <= R; ++i) first[i] = ask();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      there[i] = request(first[i], i);
      commit();
    }
    next = first[R];
  }
  int total = 0;
  for (int r = walk.r0; r < walk.r1; ++r) total += walk.tiles_of(r);
  int slot = 0;
  for (int kt = team; kt < total; kt += kTeams) {
    const int st = kt % NS, before = kt - NS;  // the tile that was there
    asm volatile("cp.async.wait_group %0;" ::"n"(R - 1) : "memory");
    // The first tile that a product has to make room for: no product starts before the row pass has ended, however
    // long that takes, so the bounded wait starts then.
    if (COLS && before >= 0 && before < kTeams) wait_for_previous_kernel();
    if (before >= 0 && !warp_wait(&mt.k_empty[before & 1], (before >> 1) & 1, abort_flag)) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      return false;
    }
    constexpr int kAtOnce = C::kIts < 8 ? C::kIts : 8;
#pragma unroll
    for (int i0 = 0; i0 < C::kIts; i0 += kAtOnce) {
      uint4 kr[kAtOnce];
#pragma unroll
      for (int it = 0; it < kAtOnce; ++it)
        kr[it] = *reinterpret_cast<const uint4*>(raw + slot * C::kRawBytes + (i0 + it) * C::kRowsIt * D);
      store_rows<D, FMT, kAtOnce>(smem + C::kOffK + st * C::kOpBytes, kr, 32 * w + i0 * C::kRowsIt, lane);
    }
    // (valid[kt % 8] of tile kt - 8 has been read: the product of kt - 4 is done, which that tile's
    // group issued behind it)
    if (lane == 0) mt.valid[kt & 7][w] = there[0];
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&mt.k_full[kt & 3]);
#pragma unroll
    for (int q = 0; q + 1 < R; ++q) there[q] = there[q + 1];
    there[R - 1] = request(next, slot);
    commit();
    next = ask();
    slot = slot + 1 == R ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  return true;
}

// Eight rows of the Q tiles: fp16 as it is, bf16 scaled by a power of two; the sign of the
// logit factor goes into Q; rows past RC are zero.
template <int D, int DT>
__device__ __forceinline__ void load_q(const ChunkParams& p, Meta& mt, uint8_t* smem, const ChunkRequest& req, int g,
                                       int row0, int first, int RC, uint32_t flip, int lane) {
  constexpr int V = D / 32;  // elements per lane
  constexpr int kAtOnce = 8;
  const int e = lane * V;
  uint8_t* sQ = smem + Cfg<D>::kOffQ + (first / kM) * Cfg<D>::kOpBytes;
  uint32_t w[kAtOnce][V / 2];
  // (rows past RC read the last one)
  RowAt at = row_at(p, row0 + min(first, RC - 1));
  const uint16_t* next = p.q + (int64_t)(req.row0 + at.token) * p.q_st + (int64_t)(g * p.G + at.head) * p.q_sh + e;
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const uint16_t* src = next;
    if (first + k + 1 < RC) {
      const bool wrap = ++at.head == p.G;
      if (wrap) at.head = 0;
      next += wrap ? p.q_st - (p.G - 1) * p.q_sh : p.q_sh;
    }
    if constexpr (V == 2)
      w[k][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
    else if constexpr (V == 4)
      *reinterpret_cast<uint2*>(w[k]) = __ldg(reinterpret_cast<const uint2*>(src));
    else
      *reinterpret_cast<uint4*>(w[k]) = __ldg(reinterpret_cast<const uint4*>(src));
  }
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int r = (first + k) % kM;
    const bool live = first + k < RC;
    float back = 1.f;
    if (DT == FP8KV_DTYPE_BF16) {
      uint32_t top = 0u;  // as integers: a NaN is larger than every number, and is not dropped
#pragma unroll
      for (int i = 0; i < V / 2; ++i) top = max(top, max((w[k][i] << 16) & 0x7FFFFFFFu, w[k][i] & 0x7FFF0000u));
      const RowScale rs = row_scale_bf16(__uint_as_float(__reduce_max_sync(0xffffffffu, top)));
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        w[k][i] = pack_half2(__uint_as_float(w[k][i] << 16) * rs.to_f16, __uint_as_float(w[k][i] & 0xFFFF0000u) * rs.to_f16);
      back = rs.back;
    }
    if (lane == 0) mt.back[first + k] = back;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[k][i] = live ? w[k][i] ^ flip : 0u;
    uint8_t* dst = sQ + (e / 64) * (kM * 128) + r * 128 + ((((e % 64) / 8) ^ (r & 7)) * 16) + (e % 8) * 2;
    if constexpr (V == 2)
      *reinterpret_cast<uint32_t*>(dst) = w[k][0];
    else if constexpr (V == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[k][0], w[k][1]);
    else
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
  }
}

// Sum of 2^(c S - m) / l over kCols columns.  The quotient goes into the exponent, as m + log2 l: a
// value that all lanes read costs a cycle of shared memory per warp and word, and three of them
// for each column (factor, maximum, 1 / sum) took 3100 cycles of a tile of 256 x 128.
// FAR: logits so large that the product is rounded before the maximum is taken off, as it was when the row's
// sum was found, and that the sum of m and log2 l would lose of the latter (kFar).  MASKED: of
// the columns whose rows see position t alone.  ONE: all rows have the factor c1.
template <bool MASKED, bool FAR, bool ONE>
__device__ __forceinline__ float column_sum(const uint32_t (&x)[kCols], const Meta& mt, int r0, int t, float c1) {
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int k = 0; k < kCols; k += 4) {
    const float4 c = ONE ? make_float4(c1, c1, c1, c1) : *reinterpret_cast<const float4*>(mt.c + r0 + k);
    float2 e0, e1, i0 = make_float2(1.f, 1.f), i1 = make_float2(1.f, 1.f);
    const float s0 = __uint_as_float(x[k]), s1 = __uint_as_float(x[k + 1]), s2 = __uint_as_float(x[k + 2]),
                s3 = __uint_as_float(x[k + 3]);
    if (FAR) {
      // (scalar: a packed product and sum came out as one fma)
      const float4 m = *reinterpret_cast<const float4*>(mt.m + r0 + k), inv = *reinterpret_cast<const float4*>(mt.inv + r0 + k);
      e0 = make_float2(__fadd_rn(__fmul_rn(s0, c.x), m.x), __fadd_rn(__fmul_rn(s1, c.y), m.y));
      e1 = make_float2(__fadd_rn(__fmul_rn(s2, c.z), m.z), __fadd_rn(__fmul_rn(s3, c.w), m.w));
      i0 = make_float2(inv.x, inv.y);
      i1 = make_float2(inv.z, inv.w);
    } else {
      const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(mt.ml + r0 + k);
      e0 = unpair(fma2(pair(s0, s1), pair(c.x, c.y), m.x));
      e1 = unpair(fma2(pair(s2, s3), pair(c.z, c.w), m.y));
    }
    if (MASKED) {
      const int4 hi = *reinterpret_cast<const int4*>(mt.hi + r0 + k);
      // neither a NaN logit nor a NaN sum of rows that do not see the position
      if (t >= hi.x) e0.x = -INFINITY, i0.x = 0.f;
      if (t >= hi.y) e0.y = -INFINITY, i0.y = 0.f;
      if (t >= hi.z) e1.x = -INFINITY, i1.x = 0.f;
      if (t >= hi.w) e1.y = -INFINITY, i1.y = 0.f;
    }
    const uint64_t p0 = pair(fast_exp2(e0.x), fast_exp2(e0.y)), p1 = pair(fast_exp2(e1.x), fast_exp2(e1.y));
    sum[0] = FAR ? fma2(p0, pair(i0.x, i0.y), sum[0]) : add2(p0, sum[0]);
    sum[1] = FAR ? fma2(p1, pair(i1.x, i1.y), sum[1]) : add2(p1, sum[1]);
  }
  const float2 s = unpair(add2(sum[0], sum[1]));
  return s.x + s.y;
}

// -(m + log2 l) of a row: the exponent of l joins the whole m exactly, the rest is below 1/2, so that
// one rounding is left (half an ulp of m + log2 l: 2^-20 at 2^4, 7e-7 of the row's weights; 2^-18 at kFar).
__device__ __forceinline__ float folded(const Norm& n) {
  if (n.inv == 0.f) return -INFINITY;  // (nothing seen)
  const uint32_t u = __float_as_uint(n.inv);
  int e = (int)(u >> 23) - 127;
  if (n.inv != n.inv || (u >> 23) == 0u || (u >> 23) == 255u) return n.inv != n.inv ? n.inv : log2f(n.inv) - n.m;
  float f = __uint_as_float((u & 0x7FFFFFu) | 0x3F800000u);  // 1 / l = 2^e f
  if (f > 1.41421356f) {
    f *= 0.5f;
    ++e;
  }
  return ((float)e - n.m) + log2f(f);
}

// Logits for which the rounded products count.
__device__ __forceinline__ void scale(uint32_t (&x)[kCols], float c) {
#pragma unroll
  for (int k = 0; k < kCols; ++k) x[k] = __float_as_uint(__fmul_rn(__uint_as_float(x[k]), c));
}

template <int D, int FMT, int DT, bool COLS>
__global__ void __launch_bounds__(kThreadsT, 1) score_tile(const __grid_constant__ ScoreParams sp) {
  using C = Cfg<D>;
  constexpr int NS = C::kStages, ROWS = C::kRows;
  const ChunkParams& p = sp.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Meta& mt = *reinterpret_cast<Meta*>(smem + C::kOffMeta);
  float* acc = reinterpret_cast<float*>(smem + C::kOffMeta + kMetaHead);  // [row tile][position of the CTA]
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int64_t plane = (int64_t)p.total_q * p.Hq;

  // (the column pass prepares everything that does not need the rows' sums while the row pass ends)
  if (!COLS) let_next_kernel_start();
  // ------------------------------------------------------ what this CTA has
  int b, g, s = 0, S = p.S;  // S: partitions of the rows' sums
  Walk walk;
  ChunkRequest req;
  if (sp.per_head > 0) {
    g = blockIdx.x % p.Hkv;
    Share share;
    if (!share_of<false>(p, sp.per_head, blockIdx.x / p.Hkv, lane, share)) {
      if (COLS) leave_in_order();
      return;
    }
    b = share.b;
    s = share.s;
    S = share.parts;
    req = chunk_request(p, b);
    walk.r0 = 0;
    walk.r1 = 1;
    walk.u0 = share.s * share.T * kT;  // (no more partitions than tiles)
    walk.u1 = (int)min((int64_t)walk.u0 + (int64_t)share.T * kT, (int64_t)req.kv);
  } else if (COLS) {
    b = div_hkv(p, blockIdx.x);
    g = blockIdx.x - b * p.Hkv;
    req = chunk_request(p, b);
    walk.u0 = (int)min((int64_t)blockIdx.z * sp.col_part, (int64_t)INT_MAX);  // (the first, longest ones start first)
    walk.u1 = (int)min((int64_t)walk.u0 + sp.col_part, (int64_t)req.kv);
    if (req.n <= 0 || walk.u0 >= req.kv) {
      leave_in_order();
      return;
    }
    // the row blocks that see anything here, and this group's share of them
    const int base = req.kv - req.n, blocks = (req.n * p.G + ROWS - 1) / ROWS;
    const int first = max(0, walk.u0 - base) * p.G / ROWS, share = (blocks - first + sp.groups - 1) / sp.groups;
    walk.r0 = min(first + (int)blockIdx.y * share, blocks);
    walk.r1 = min(walk.r0 + share, blocks);
    s = blockIdx.y;
    if (walk.r0 >= walk.r1) {  // (only one of several groups)
      float* to = sp.partial + (((int64_t)s * p.B + b) * p.Hkv + g) * p.max_kv_len;
      for (int t = walk.u0 + tid; t < walk.u1; t += kThreadsT) to[t] = 0.f;
      leave_in_order();
      return;
    }
  } else {
    TileWork work;
    g = blockIdx.x % p.Hkv;
    s = blockIdx.y;
    if (!locate(p, ROWS, blockIdx.x / p.Hkv, lane, work)) return;
    b = work.b;
    req = chunk_request(p, b);
    if (req.n * p.G <= work.row0 || work.row0 < 0) return;
    walk.r0 = work.row0 / ROWS;
    walk.r1 = walk.r0 + 1;
    walk.u0 = (int)min((int64_t)s * sp.stat_part, (int64_t)INT_MAX);
  }
  walk.base = req.kv - req.n;
  walk.G = p.G;
  walk.rows = ROWS;
  walk.n = req.n;
  const int RC0 = min(ROWS, req.n * p.G - walk.r0 * ROWS);  // rows of the first block
  auto vec_of = [&](int rr) { return (int64_t)(req.row0 + token_at(p, rr)) * p.Hq + g * p.G + row_at(p, rr).head; };
  if (!COLS && sp.per_head == 0) {
    const int U = max(walk.last_of(walk.r0), 0);
    walk.u1 = (int)min((int64_t)walk.u0 + sp.stat_part, (int64_t)U);
    if (walk.u0 >= walk.u1) {
      for (int r = tid; r < RC0; r += kThreadsT)
        p.ml[s * plane + vec_of(walk.r0 * ROWS + r)] = make_float2(kNoMax, 0.f);
      return;
    }
  }
  // row tiles in use; one alone only where there is no second row block (D = 256: always one)
  const int nq = __shfl_sync(0xffffffffu, C::kNQ == 2 && (walk.r1 - walk.r0 > 1 || RC0 > kM) ? 2 : 1, 0);
  // sums of several row tiles meet in `acc` (in shares of any length: each has its place in `partial`)
  const bool gather = COLS && sp.per_head == 0 && (nq == 2 || walk.r1 - walk.r0 > 1);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&mt.k_empty[i], nq);
    for (int i = 0; i < 4; ++i) mbar_init(&mt.k_full[i], 4);  // one lane of each decoder warp
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&mt.s_full[i], 1);
      mbar_init(&mt.s_empty[i], 4);  // one lane of each of the group's warps
      mbar_init(&mt.drain[i], 1);
    }
    mt.abort = 0u;
    mbar_init_fence();
  }
  if (warp == 0) {
    tmem_alloc(&mt.tmem, 512);
    tmem_relinquish();
  }
  if (gather)
    for (int i = tid; i < 2 * kScoreAccTokens; i += kThreadsT) acc[i] = 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, mt.tmem, 0);
  volatile uint32_t* const abort_flag = &mt.abort;
  const float ks = p.k_scale_dev ? *p.k_scale_dev : p.k_scale;
  const float cf = p.softmax_scale * ks * kLog2e;  // base-2 logit factor
  bool ok = true;

  if (warp < 4 * kGroups) {
    const int w = warp >> 2, wl = warp & 3;             // group, warp of it
    const int tile = nq == 2 ? w & 1 : 0;               // the group's row tile
    const int j0 = nq == 2 ? w >> 1 : w, j_step = nq == 2 ? 2 : 4;  // ... and K tiles of a row block
    const uint32_t tS = tmem + w * 128 + ((uint32_t)(32 * wl) << 16);
    const uint32_t idesc = idesc_f16_f32(kM, kT, false, false);
    const uint64_t qdesc = smem_desc(smem_u32(smem + C::kOffQ + tile * C::kOpBytes), 16, 1024, kSw128);
    const uint64_t kdesc = smem_desc(smem_u32(smem + C::kOffK), 16, 1024, kSw128);
    // The product with K tile kt, by the group's first warp.  A group may be several stages behind the
    // decoders, and a barrier's parity tells two neighbouring phases apart, no more: of the
    // barrier for every fourth tile, the phase before this one (kt - 4) is one that the group, or a
    // row block that all groups are past, has used.
    auto issue = [&](int kt) {
      ok = ok && warp_wait(&mt.k_full[kt & 3], (kt >> 2) & 1, abort_flag);
      if (!ok) return;
      tc_fence_after();
      const uint64_t kd = kdesc + (uint64_t)(((kt % NS) * C::kOpBytes) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t step = (uint64_t)(((kk / 4) * (kM * 128) + (kk % 4) * 32) >> 4);
          mma_ss(tmem + w * 128, (COLS ? kd : qdesc) + step, (COLS ? qdesc : kd) + step, idesc, kk > 0);
        }
        mma_commit(&mt.s_full[w]);
        mma_commit(&mt.k_empty[kt & 1]);
      }
      __syncwarp();
    };
    int ktb = 0, uses = 0;                              // K tiles of earlier row blocks; products of this group so far
    for (int rb = walk.r0; rb < walk.r1; ++rb) {
      // ---------------------------------------------------- Q, and what is known of its rows
      // (every group has waited for its products of the last block)
      const int row0 = rb * ROWS, RC = min(ROWS, req.n * p.G - row0);
      named_bar_sync(1, kEpilogue);
      for (int k = 0; k < nq; ++k)
        load_q<D, DT>(p, mt, smem, req, g, row0, (warp * nq + k) * 8, RC, cf < 0.f ? 0x80008000u : 0u, lane);
      fence_proxy_async_smem();
      named_bar_sync(1, kEpilogue);
      if (COLS && rb == walk.r0) wait_for_previous_kernel();
      if (tid < nq * kM) {
        // (not 0, so that c * -inf stays -inf; nor NaN: a NaN scale goes into the rows' sums)
        mt.c[tid] = fmaxf(fabsf(cf) * mt.back[tid], 1e-30f);
        const bool live = tid < RC;
        mt.hi[tid] = live ? max(walk.base + token_at(p, row0 + tid) + 1, 0) : 0;
        if (COLS) {
          const Norm n = live ? join_norm(p.ml, plane, vec_of(row0 + tid), S) : Norm{0.f, 0.f};
          mt.m[tid] = -n.m;
          mt.inv[tid] = n.inv;
          mt.ml[tid] = folded(n);
        }
      }
      named_bar_sync(1, kEpilogue);
      const int n_tiles = walk.tiles_of(rb);
      if (wl == 0 && j0 < n_tiles) issue(ktb + j0);
      // the group's rows: the least that one sees; columns: whether logits are past kFar
      const int mine = tile * kM + 32 * wl + lane;      // rows: this thread's
      int hi = mine < RC ? mt.hi[mine] : INT_MAX;       // rows past RC: everything, dropped at the end
      const float c = mt.c[mine];
      bool far_cols = false;
      if (COLS) {
        float top = 0.f;
        hi = INT_MAX;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi = min(hi, mt.hi[tile * kM + 32 * i + lane]);
          top = fmaxf(top, fabsf(mt.m[tile * kM + 32 * i + lane]));
        }
        far_cols = __any_sync(0xffffffffu, top >= kFar);
      }
      const int hi_min = __reduce_min_sync(0xffffffffu, hi);
      constexpr bool kOne = DT == FP8KV_DTYPE_F16;      // (bf16 rows have scales of their own)
      // rows: a whole number near the largest logit; the sum, and what its additions rounded off (a row has
      // up to 2^26 / 32 of them)
      float m = 0.f, l = 0.f, l_rest = 0.f;
      bool started = false;                             // ... a logit above -inf was seen
      bool far = false;                                 // some row of the warp has logits past kFar: products are rounded
                                                        // before the maximum is taken off
      for (int j = j0; j < n_tiles; j += j_step) {
        const int kt = ktb + j, parity = uses & 1;
        ok = ok && warp_wait(&mt.s_full[w], parity, abort_flag);
        ++uses;
        if (!ok) break;
        tc_fence_after();
        const int v0 = walk.u0 + j * kT;
        const uint4 there = *reinterpret_cast<const uint4*>(mt.valid[kt & 7]);
        const bool masked = v0 + kT > hi_min || (!COLS && (there.x & there.y & there.z & there.w) != 0xFFFFFFFFu);
        const int t = v0 + 32 * wl + lane;              // columns: this thread's position
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < kT / kCols; ++h) {
          uint32_t x[kCols];
          tmem_ld32(tS + kCols * h, x);
          if (h == kT / kCols - 1) {
            // S is read: the next product may be written over it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&mt.s_empty[w]);
            if (wl == 0 && j + j_step < n_tiles) {
              ok = warp_wait(&mt.s_empty[w], parity, abort_flag);
              issue(kt + j_step);
            }
          }
          if (COLS) {
            const int r0 = tile * kM + kCols * h;
            if (far_cols)
              sum += masked ? column_sum<true, true, false>(x, mt, r0, t, c) : column_sum<false, true, false>(x, mt, r0, t, c);
            else
              sum += masked ? column_sum<true, false, kOne>(x, mt, r0, t, c) : column_sum<false, false, kOne>(x, mt, r0, t, c);
          } else {
            if (masked) {
              // logits that the row does not see become -inf (a NaN among them too)
              const uint32_t vis =
                  (h == 0 ? there.x : h == 1 ? there.y : h == 2 ? there.z : there.w) & below(hi - v0 - kCols * h);
#pragma unroll
              for (int k = 0; k < kCols; ++k) x[k] = ((vis >> k) & 1u) ? x[k] : 0xFF800000u;
            }
            // Sum of the weights over the maximum so far: in FP32 it may be any near one, so it moves only
            // when the sum has grown past 2^40 (or is not a number), and no maximum is looked for else.
            auto weights = [&]() {
              const uint64_t c2 = far ? pair(1.f, 1.f) : pair(c, c), sh2 = pair(-m, -m);
              uint64_t part[2] = {0ull, 0ull};
#pragma unroll
              for (int k = 0; k < kCols; k += 2) {
                const float2 e = unpair(fma2(pair(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), c2, sh2));
                part[(k / 2) & 1] = add2(part[(k / 2) & 1], pair(fast_exp2(e.x), fast_exp2(e.y)));
              }
              const float2 y = unpair(add2(part[0], part[1]));
              return y.x + y.y;
            };
            if (far) scale(x, c);
            float y = started ? weights() : INFINITY;
            if (__any_sync(0xffffffffu, !(y < 0x1p40f))) {
              float top = -INFINITY;  // (a NaN is passed over: it makes the sum NaN)
#pragma unroll
              for (int k = 0; k < kCols; ++k) top = fmaxf(top, __uint_as_float(x[k]));
              top = far ? top : __fmul_rn(top, c);
              const float n = top == -INFINITY ? m : started ? fmaxf(m, ceilf(top)) : ceilf(top);
              if (started) {
                const float a = exp2_whole(m - n);
                l *= a;
                l_rest *= a;
              }
              m = n;
              started |= top != -INFINITY;
              if (!far && __any_sync(0xffffffffu, fabsf(m) >= kFar)) {
                far = true;
                scale(x, c);
              }
              // (before the first logit above -inf m is 0, and what is added 0, or NaN for a NaN logit)
              y = weights();
            }
            two_sum_acc(l, l_rest, y);
          }
        }
        if (COLS && t < walk.u1) {
          if (!(((wl == 0 ? there.x : wl == 1 ? there.y : wl == 2 ? there.z : there.w) >> lane) & 1u)) sum = 0.f;
          if (gather)
            acc[tile * kScoreAccTokens + t - walk.u0] += sum;
          else if (sp.groups == 1)
            write_score(sp, b, g, t, walk.base, sum);
          else {
            const int64_t row_len = (int64_t)p.B * p.Hkv * p.max_kv_len;
            float* to = sp.partial + ((int64_t)b * p.Hkv + g) * p.max_kv_len + t;
            to[(sp.per_head > 0 ? tile : s) * row_len] = sum;
            if (sp.per_head > 0 && nq == 1) to[row_len] = 0.f;  // (a request without a second row tile)
          }
        }
      }
      ktb += n_tiles;
      if (!COLS) {
        l += l_rest;
        if (cf != cf && l != 0.f) l = cf;
        if (!started) m = kNoMax;
        // the groups' shares of the positions
        const int heirs = nq;  // groups 0 (and 1) take over
        if (w >= heirs) mt.other[w - 1][32 * wl + lane] = make_float2(m, l);
        named_bar_sync(1, kEpilogue);
        if (w < heirs) {
          float M = m;
          for (int q = w + heirs; q < kGroups; q += heirs) M = fmaxf(M, mt.other[q - 1][32 * wl + lane].x);
          float L = l != 0.f ? l * part_weight(m, M) : 0.f;
          for (int q = w + heirs; q < kGroups; q += heirs) {
            const float2 y = mt.other[q - 1][32 * wl + lane];
            if (y.y != 0.f) L = fmaf(y.y, part_weight(y.x, M), L);
          }
          if (ok && mine < RC) p.ml[s * plane + vec_of(row0 + mine)] = make_float2(M, L);
        }
      }
    }
    if (COLS && !gather && sp.groups > 1 && sp.per_head == 0) {  // positions that none of the block's rows sees
      float* to = sp.partial + (((int64_t)s * p.B + b) * p.Hkv + g) * p.max_kv_len;
      for (int t = walk.u0 + walk.tiles_of(walk.r0) * kT + tid; t < walk.u1; t += kEpilogue) to[t] = 0.f;
    }
    if (gather) {
      named_bar_sync(1, kEpilogue);
      if (ok)
        for (int t = walk.u0 + tid; t < walk.u1; t += kEpilogue) {
          const float sum = acc[t - walk.u0] + acc[kScoreAccTokens + t - walk.u0];
          if (sp.groups == 1)
            write_score(sp, b, g, t, walk.base, sum);
          else
            sp.partial[(((int64_t)s * p.B + b) * p.Hkv + g) * p.max_kv_len + t] = sum;
        }
    }
    if (wl == 0) {
      // every UMMA issued must be done before TMEM is freed
      if (elect_one()) mma_commit(&mt.drain[w]);
      __syncwarp();
      mbar_wait_plain(&mt.drain[w], 0, kPolls);
      __syncwarp();
    }
  } else {
    ok = decode_k<D, FMT, COLS>(p, mt, smem, b, g, walk, (warp >> 2) - kGroups, warp & 3, lane);
  }
  if (!ok) set_status(p.status, FP8KV_STATUS_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sums of the row groups: a thread per position.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) score_sum(const __grid_constant__ ScoreParams sp) {
  const ChunkParams& p = sp.c;
  const int b = div_hkv(p, blockIdx.y), g = blockIdx.y - b * p.Hkv;
  const ChunkRequest req = chunk_request(p, b);
  const int t = (int)min((int64_t)blockIdx.x * kSumThreads + threadIdx.x, (int64_t)INT_MAX);
  if (req.n <= 0 || t >= req.kv) return;
  const int64_t step = (int64_t)p.B * p.Hkv * p.max_kv_len;
  const float* from = sp.partial + ((int64_t)b * p.Hkv + g) * p.max_kv_len + t;
  float sum = 0.f;
  for (int i = 0; i < sp.groups; ++i) sum += from[i * step];
  write_score(sp, b, g, t, req.kv - req.n, sum);
}

template <int D, int FMT, int DT>
cudaError_t run(const fp8kv_cache_score_plan_t*, const ScoreParams& p, cudaStream_t st) {
  auto rows = score_tile<D, FMT, DT, false>;
  auto cols = score_tile<D, FMT, DT, true>;
  constexpr int smem = Cfg<D>::kSmem;
  static DeviceOnce once;
  cudaError_t e = once.run([&] {
    const cudaError_t x = cudaFuncSetAttribute(rows, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return x != cudaSuccess ? x : cudaFuncSetAttribute(cols, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  const int pairs = p.c.B * p.c.Hkv;
  if (p.per_head > 0) {
    rows<<<dim3(p.per_head * p.c.Hkv), kThreadsT, smem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_dependent(cols, dim3(p.per_head * p.c.Hkv), kThreadsT, smem, st, p);
  } else {
    rows<<<dim3(p.c.row_tiles * p.c.Hkv, p.c.S), kThreadsT, smem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int parts = (int)(((int64_t)p.c.max_kv_len + p.col_part - 1) / p.col_part);
    e = launch_dependent(cols, dim3(pairs, p.groups, parts), kThreadsT, smem, st, p);
  }
  if (e != cudaSuccess || p.groups == 1) return e;
  score_sum<<<dim3((unsigned)((p.c.max_kv_len + kSumThreads - 1) / kSumThreads), pairs), kSumThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t pick(const fp8kv_cache_score_plan_t* plan, const ScoreParams& p, cudaStream_t st) {
  constexpr int E4 = FP8KV_KV_E4M3, E5 = FP8KV_KV_E5M2, F16 = FP8KV_DTYPE_F16, BF16 = FP8KV_DTYPE_BF16;
  if (plan->kv_format == E5)
    return plan->dtype == BF16 ? run<D, E5, BF16>(plan, p, st) : run<D, E5, F16>(plan, p, st);
  return plan->dtype == BF16 ? run<D, E4, BF16>(plan, p, st) : run<D, E4, F16>(plan, p, st);
}

}  // namespace

cudaError_t launch_score_tile(const fp8kv_cache_score_plan_t* plan, const ScoreParams& p, cudaStream_t st) {
  switch (plan->head_dim) {
    case 64: return pick<64>(plan, p, st);
    case 128: return pick<128>(plan, p, st);
    default: return pick<256>(plan, p, st);
  }
}

}  // namespace fp8kv
