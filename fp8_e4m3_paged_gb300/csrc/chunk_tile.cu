// Chunk attention for many query vectors: tcgen05 tiles of 128 vectors by 128
// positions.
//
// The query heads of one KV head and the new tokens of one request are packed
// into rows (token * G + head), so a tile is full whatever the group size and
// one decode of K and V serves all of them.  A CTA owns 256 rows (two row
// tiles; 128 rows for D = 256) of one request and KV head, and one partition
// of the positions that its rows see.  Warp roles:
//   warps 0-3, 4-7   softmax of row tile 0 and 1 (thread = row = TMEM lane);
//                    D = 256: warps 0-3 only, and warps 4-7 decode K;
//   warps 8-11       decode K and V (D = 256: V): FP8 rows, requested one tile
//                    ahead, into swizzled fp16 operand tiles;
//   warp 12          TMEM, and every UMMA.
// Per tile j and row tile q:  S_q = Q_q . K_j^T (M 128, N 128),
// P_q = 2^(s - m + 7) as fp16 over S_q in TMEM, O_q += P_q . V_j (A from TMEM).
// Two row tiles alternate: while one's softmax runs, the tensor core works on
// the other's S and O.  For D = 256 two S buffers of the one row tile do the
// same: QK of tile j+1 is issued before PV of tile j.
// TMEM: S at columns 0 and 128, O at 256 (256 columns).
//
// Every wait is bounded (see split_tc_kernel.cuh): a wait that gives up sets the
// CTA's abort flag and FP8KV_STATUS_TIMEOUT, every role stops, and the issued
// UMMAs are drained before TMEM is freed.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk_common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace fp8kv {
namespace {

using namespace tc;

constexpr int kT = kChunkTileTokens;
constexpr int kM = 128;                  // rows per tile
constexpr int kTileThreads = 13 * 32;
constexpr int kMmaWarp = 12;
constexpr int kStagesMax = 4;
constexpr uint32_t kPolls = 1u << 20;    // polls per wait

template <int D>
struct TileCfg {
  static constexpr int kNQ = D == 256 ? 1 : 2;
  static constexpr int kStages = D == 256 ? 1 : D == 128 ? 2 : 4;  // K stages, and V stages
  static constexpr int kOpBytes = kT * D * 2;
  static constexpr int kCh = D / 16;          // 16-byte pieces of an FP8 row
  static constexpr int kRowsIt = 32 / kCh;    // rows a warp moves at a time
  static constexpr int kParts = D == 256 ? 2 : 1;       // a tile's rows are staged in so many parts (shared memory)
  static constexpr int kIts = 32 / kRowsIt / kParts;    // times, for its rows of a part
  static constexpr int kRawBytes = 2 * kT * D / kParts; // staged FP8 rows of K and V
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kNQ * kM * D * 2;
  static constexpr int kOffV = kOffK + kStages * kOpBytes;
  static constexpr int kOffRaw = kOffV + kStages * kOpBytes;  // FP8 K rows, then V rows
  static constexpr int kOffMeta = kOffRaw + kRawBytes;
  static constexpr int kSmem = kOffMeta + 2048 + 1024;  // meta, alignment
  static constexpr uint32_t kColO = 256;
  static_assert(kNQ * D <= 256 && kSmem <= 232448, "TMEM and shared memory");
};

struct TileMeta {
  uint64_t q_full, drain;
  uint64_t k_full[kStagesMax], k_empty[kStagesMax], v_full[kStagesMax], v_empty[kStagesMax];
  uint64_t s_full[2], p_ready[2], o_all[2];  // o_all: a row tile's last PV is done
  uint64_t o_done;                           // D = 256: PV(j) is done, every tile but the last
  uint32_t valid[8][4];  // per tile (j % 8): positions whose block is in range
  uint32_t tmem, abort, vbad;
  float back[2 * kM];    // inverse row scales
};
static_assert(sizeof(TileMeta) <= 2048, "meta block");

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

// Request and first packed row of this CTA: tiles count over the requests in
// order, taken from the last (a request's last rows see the most positions,
// so the longest work starts first).
struct TileWork {
  int b, row0;
};
__device__ __forceinline__ int tiles_of(const ChunkParams& p, int b, int rows, bool& bad) {
  if (b >= p.B) return 0;
  const ChunkRequest r = chunk_request(p, b);
  bad |= r.bad;
  return (r.n * p.G + rows - 1) / rows;
}
__device__ __forceinline__ bool locate(const ChunkParams& p, int rows, int lane, TileWork& w) {
  int total = 0;
  bool bad = false;
  for (int b0 = 0; b0 < p.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, tiles_of(p, b0 + lane, rows, bad));
  if (bad && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 32)
    set_status(p.status, FP8KV_STATUS_BAD_LEN);
  int idx = total - 1 - (int)blockIdx.x;
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

// A decoder lane's 16-byte pieces of one tile part (piece lane % kCh of rows
// it * kRowsIt + lane / kCh of the warp's rows of the part).  They wait in shared memory,
// in places that only this lane writes (cp.async) and reads, so no barrier is
// needed; in registers, K and V in flight would take 64.  The copies are
// unconditional: rows without a place read the pool's first one.
template <int D>
__device__ __forceinline__ void stage_rows(const uint8_t* base, int64_t off, int part, int lane, uint8_t* raw) {
  using C = TileCfg<D>;
#pragma unroll
  for (int it = 0; it < C::kIts; ++it) {
    const int64_t o = __shfl_sync(0xffffffffu, off, (part * C::kIts + it) * C::kRowsIt + lane / C::kCh);
    cp_async16(raw + (it * 32 + lane) * 16, base + o + (lane % C::kCh) * 16);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int D>
__device__ __forceinline__ void take_rows(const uint8_t* raw, int lane, uint4 (&w)[TileCfg<D>::kIts]) {
  using C = TileCfg<D>;
#pragma unroll
  for (int it = 0; it < C::kIts; ++it) w[it] = *reinterpret_cast<const uint4*>(raw + (it * 32 + lane) * 16);
}

// ... and as fp16 in the operand tile: 64-column blocks of kT rows of 128
// bytes, 16-byte chunk c of row r at c ^ (r % 8).  Odd column blocks store
// their two chunks in the other order, so that eight lanes hit eight banks.
template <int D, int FMT>
__device__ __forceinline__ void store_rows(uint8_t* op, const uint4 (&w)[TileCfg<D>::kIts], int row_base, int lane) {
  using C = TileCfg<D>;
  const int c = lane % C::kCh, db = c / 4, h0 = (c % 4) * 2;
  const bool swap = db & 1;
  const int first = swap ? h0 + 1 : h0, second = swap ? h0 : h0 + 1;
#pragma unroll
  for (int it = 0; it < C::kIts; ++it) {
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

// V pieces before they are stored: zero for rows whose block is out of range or that
// lie past the partition (their weight is 0, and 0 * NaN would not be; K rows
// need not, their logits are masked), and non-finite codes as zero (returns
// true if there were any).  ok: the part's rows from bit 0 on.
template <int D, int FMT>
__device__ __forceinline__ bool clean_v(uint4 (&w)[TileCfg<D>::kIts], uint32_t ok, int lane) {
  using C = TileCfg<D>;
  constexpr bool e5 = FMT == FP8KV_KV_E5M2;
  if (ok != 0xFFFFFFFFu) {
#pragma unroll
    for (int i = 0; i < C::kIts; ++i)
      if (!((ok >> (i * C::kRowsIt + lane / C::kCh)) & 1u)) w[i] = make_uint4(0, 0, 0, 0);
  }
  uint32_t any = 0u;
#pragma unroll
  for (int i = 0; i < C::kIts; ++i) any |= nonfinite_codes(w[i], e5);
  if (any == 0u) return false;
#pragma unroll
  for (int i = 0; i < C::kIts; ++i)
    w[i] = make_uint4(zap_nonfinite(w[i].x, e5), zap_nonfinite(w[i].y, e5), zap_nonfinite(w[i].z, e5),
                      zap_nonfinite(w[i].w, e5));
  return true;
}

// Decoders: K, V or both streams of every tile.
template <int D, int FMT, bool DO_K, bool DO_V>
__device__ __forceinline__ bool decode_tiles(const ChunkParams& p, TileMeta& mt, uint8_t* smem, int b, int g, int u0,
                                             int u1, int n_tiles, const ChunkSpan& span, int w, int lane) {
  using C = TileCfg<D>;
  constexpr int NS = C::kStages, PARTS = C::kParts, PART_ROWS = 32 / PARTS;
  volatile uint32_t* const abort_flag = &mt.abort;
  const uint8_t* kbase = p.k_cache + g * p.ksh;
  const uint8_t* vbase = p.v_cache + g * p.vsh;
  // Position 32 w + lane of a tile: its block id is requested one tile before
  // the place is needed, so that nothing waits for that load either.
  int blk = -1, slot = 0;
  bool in = false;
  auto ask = [&](int j) {
    const int v = u0 + j * kT + 32 * w + lane;
    in = v < u1;
    blk = -1;
    if (in) {
      const int pos = span.position(v), page = div_page(pos, p.page_size, p.page_div);
      slot = pos - page * p.page_size;
      blk = __ldg(p.block_table + (int64_t)b * p.bt_stride + page);
    }
  };
  int64_t koff = 0, voff = 0;
  uint32_t ok_next = 0u;
  auto find = [&]() {
    const bool ok = blk >= 0 && blk < p.num_kv_blocks;
    if (DO_K && in && !ok) set_status(p.status, FP8KV_STATUS_BAD_BLOCK);
    if (DO_K) koff = ok ? blk * p.ksb + (int64_t)slot * p.kst : 0;
    if (DO_V) voff = ok ? blk * p.vsb + (int64_t)slot * p.vst : 0;
    ok_next = __ballot_sync(0xffffffffu, ok);
  };
  uint8_t* rawk = smem + C::kOffRaw + w * (PART_ROWS * D);
  uint8_t* rawv = rawk + C::kRawBytes / 2;
  ask(0);
  find();
  if (DO_K) stage_rows<D>(kbase, koff, 0, lane, rawk);
  if (DO_V) stage_rows<D>(vbase, voff, 0, lane, rawv);
  uint32_t ok_now = ok_next;
  if (n_tiles > 1) ask(1);
  bool ok = true, bad = false;
  for (int j = 0; j < n_tiles && ok; ++j) {
    const int st = j % NS;
    const uint32_t empty_parity = ((j / NS) - 1) & 1;
    // A stage copy follows each part taken (the very last one again), so that the
    // number of copies in flight is always the same.
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      const int next = (part + 1) % PARTS;
      if (next == 0) {
        if (j + 1 < n_tiles) find();
        if (j + 2 < n_tiles) ask(j + 2);
      }
      uint4 x[C::kIts];
      if constexpr (DO_K) {
        if (DO_V)
          asm volatile("cp.async.wait_group 1;" ::: "memory");  // V's is still under way
        else
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        take_rows<D>(rawk, lane, x);
        if (part == 0 && j >= NS && !warp_wait(&mt.k_empty[st], empty_parity, abort_flag)) {
          ok = false;
          break;
        }
        store_rows<D, FMT>(smem + C::kOffK + st * C::kOpBytes, x, 32 * w + part * PART_ROWS, lane);
        if (next == 0) {
          // K(j+8) is decoded after QK(j+4) at the earliest, and that after softmax j+3
          if (lane == 0) mt.valid[j & 7][w] = ok_now;
          fence_proxy_async_smem();
          mbar_arrive(&mt.k_full[st]);
        }
        stage_rows<D>(kbase, koff, next, lane, rawk);
      }
      if constexpr (DO_V) {
        if (DO_K)
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        take_rows<D>(rawv, lane, x);
        // the part's rows from bit 0 on, no row missing above them
        constexpr uint32_t above = PARTS == 1 ? 0u : 0xFFFF0000u;
        bad |= clean_v<D, FMT>(x, (ok_now >> (part * PART_ROWS)) | above, lane);
        if (part == 0 && j >= NS && !warp_wait(&mt.v_empty[st], empty_parity, abort_flag)) {
          ok = false;
          break;
        }
        store_rows<D, FMT>(smem + C::kOffV + st * C::kOpBytes, x, 32 * w + part * PART_ROWS, lane);
        if (next == 0) {
          fence_proxy_async_smem();
          mbar_arrive(&mt.v_full[st]);
        }
        stage_rows<D>(vbase, voff, next, lane, rawv);
      }
    }
    ok_now = ok_next;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (bad) mt.vbad = 1u;
  return ok;
}

// Visibility of 32 virtual tokens v0 .. v0+31 for one row, as bits.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t sees32(const ChunkRow& r, int sk, int v0) {
  return below(r.hi - v0) & (~below(r.lo - v0) | below(sk - v0));
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Largest visible element of this thread's 128 columns of S (a NaN is passed
// over: it makes the row's sum NaN).  FULL: every column is visible.
template <bool FULL>
__device__ __forceinline__ float row_max(uint32_t tS, const uint32_t (&vis)[4]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x[32];
    tmem_ld32(tS + 32 * i, x);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float v = __uint_as_float(x[k]);
      m[(k / 2) & 3] = fmaxf(m[(k / 2) & 3], FULL || ((vis[i] >> k) & 1u) ? v : -INFINITY);
    }
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// P = 2^(c S + sh) as fp16 over S (masked columns: 0); returns the sum.
template <bool FULL>
__device__ __forceinline__ float exp_tile(uint32_t tS, const uint32_t (&vis)[4], float c, float sh) {
  const uint64_t c2 = pair(c, c), sh2 = pair(sh, sh);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x[32], y[16];
    tmem_ld32(tS + 32 * i, x);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      float2 e = unpair(fma2(pair(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), c2, sh2));
      if (!FULL) {
        e.x = ((vis[i] >> k) & 1u) ? e.x : -INFINITY;
        e.y = ((vis[i] >> (k + 1)) & 1u) ? e.y : -INFINITY;
      }
      const float p0 = fast_exp2(e.x), p1 = fast_exp2(e.y);
      sum[(k / 2) & 1] = add2(sum[(k / 2) & 1], pair(p0, p1));
      y[k / 2] = pack_half2(p0, p1);
    }
    tmem_st16(tS + 16 * i, y);  // over S columns that were read
  }
  const float2 t = unpair(add2(sum[0], sum[1]));
  return t.x + t.y;
}

template <int D, int FMT, int DT>
__global__ void __launch_bounds__(kTileThreads, 1) chunk_tile(const __grid_constant__ ChunkParams p) {
  using C = TileCfg<D>;
  constexpr int NQ = C::kNQ, ROWS = NQ * kM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TileMeta& mt = *reinterpret_cast<TileMeta*>(smem + C::kOffMeta);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y, s = blockIdx.z;

  TileWork work;
  if (!locate(p, ROWS, lane, work)) return;
  const int b = work.b;
  const ChunkRequest req = chunk_request(p, b);
  const int RC = min(ROWS, req.n * p.G - work.row0);
  if (RC <= 0 || work.row0 < 0) return;
  const int64_t plane = (int64_t)p.total_q * p.Hq;
  auto vec_of = [&](int r) {
    const int rr = work.row0 + r;
    return (int64_t)(req.row0 + rr / p.G) * p.Hq + g * p.G + rr % p.G;
  };
  const ChunkSpan span = chunk_span(p, req, work.row0 / p.G, (work.row0 + RC - 1) / p.G);
  int per = (span.U + p.S - 1) / p.S;
  per = (per + kT - 1) / kT * kT;
  const int u0 = (int)min((int64_t)s * per, (int64_t)span.U), u1 = min(span.U, u0 + per);
  if (u0 >= u1) {  // nothing to see here: an empty partition, or rows before position 0
    if (p.S > 1) {
      for (int r = tid; r < RC; r += kTileThreads) p.ml[s * plane + vec_of(r)] = make_float2(kNoMax, 0.f);
    } else {
      for (int x = tid; x < RC * (D / 8); x += kTileThreads) {
        const int rr = work.row0 + x / (D / 8);
        *reinterpret_cast<uint4*>(p.out + (int64_t)(req.row0 + rr / p.G) * p.o_st +
                                  (int64_t)(g * p.G + rr % p.G) * p.o_sh + (x % (D / 8)) * 8) = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  const int n_tiles = (u1 - u0 + kT - 1) / kT;
  const int nq = NQ == 2 && RC > kM ? 2 : 1;  // row tiles in use

  if (tid == 0) {
    mbar_init(&mt.q_full, nq * kM);
    mbar_init(&mt.drain, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&mt.k_full[i], 128);
      mbar_init(&mt.k_empty[i], 1);
      mbar_init(&mt.v_full[i], 128);
      mbar_init(&mt.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&mt.s_full[i], 1);
      mbar_init(&mt.p_ready[i], kM);
      mbar_init(&mt.o_all[i], 1);
    }
    mbar_init(&mt.o_done, 1);
    mt.abort = 0u;
    mt.vbad = 0u;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&mt.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = mt.tmem;
  volatile uint32_t* const abort_flag = &mt.abort;
  const float ks = p.k_scale_dev ? *p.k_scale_dev : p.k_scale;
  const double cd = (double)p.softmax_scale * (double)ks * 1.4426950408889634074;
  bool ok = true;

  if (warp < 4 * NQ) {
    const int q = warp >> 2;
    if (q < nq) {
      // ====================================================== Q tile
      // One warp per row: fp16 as it is, bf16 scaled by a power of two; the
      // sign of the logit factor goes into Q.
      constexpr int V = D / 32;  // elements per lane
      constexpr int kRowsAtOnce = 8;
      uint8_t* sQ = smem + C::kOffQ + q * (kM * D * 2);
      const uint32_t flip = cd < 0 ? 0x80008000u : 0u;
      const int e = lane * V;  // first element of the lane
#pragma unroll 1
      for (int k0 = 0; k0 < 32; k0 += kRowsAtOnce) {
        uint32_t w[kRowsAtOnce][V / 2];
        // all loads first, rows past RC read the last one (their results are dropped)
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k) {
          const int pr = work.row0 + min(q * kM + 32 * (warp & 3) + k0 + k, RC - 1);
          const uint16_t* src =
              p.q + (int64_t)(req.row0 + pr / p.G) * p.q_st + (int64_t)(g * p.G + pr % p.G) * p.q_sh + e;
          if constexpr (V == 2) {
            w[k][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
          } else if constexpr (V == 4) {
            *reinterpret_cast<uint2*>(w[k]) = __ldg(reinterpret_cast<const uint2*>(src));
          } else {
            *reinterpret_cast<uint4*>(w[k]) = __ldg(reinterpret_cast<const uint4*>(src));
          }
        }
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k) {
          const int r = 32 * (warp & 3) + k0 + k;
          if (DT == FP8KV_DTYPE_BF16) {
            uint32_t top = 0u;  // as integers: a NaN is larger than every number, and is not dropped
#pragma unroll
            for (int i = 0; i < V / 2; ++i) top = max(top, max((w[k][i] << 16) & 0x7FFFFFFFu, w[k][i] & 0x7FFF0000u));
            const RowScale rs = row_scale_bf16(__uint_as_float(__reduce_max_sync(0xffffffffu, top)));
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
              w[k][i] = pack_half2(__uint_as_float(w[k][i] << 16) * rs.to_f16,
                                   __uint_as_float(w[k][i] & 0xFFFF0000u) * rs.to_f16);
            if (lane == 0) mt.back[q * kM + r] = rs.back;
          }
#pragma unroll
          for (int i = 0; i < V / 2; ++i) w[k][i] ^= flip;
          uint8_t* dst = sQ + (e / 64) * (kM * 128) + r * 128 + ((((e % 64) / 8) ^ (r & 7)) * 16) + (e % 8) * 2;
          if constexpr (V == 2)
            *reinterpret_cast<uint32_t*>(dst) = w[k][0];
          else if constexpr (V == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(w[k][0], w[k][1]);
          else
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
        }
      }
      __syncwarp();
      fence_proxy_async_smem();
      mbar_arrive(&mt.q_full);

      // ====================================================== softmax
      const int rr = q * kM + 32 * (warp & 3) + lane;  // this thread's row of the CTA
      const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
      const float c = (float)(fabs(cd) * (DT == FP8KV_DTYPE_BF16 ? (double)mt.back[rr] : 1.0));
      ChunkRow row = {INT_MAX, INT_MIN};  // rows past RC: everything, dropped at the end
      if (rr < RC) row = chunk_row(p, req, span, (work.row0 + rr) / p.G);
      const int hi_min = __reduce_min_sync(0xffffffffu, row.hi), lo_max = __reduce_max_sync(0xffffffffu, row.lo);
      float m = kNoMax, l = 0.f;
      const uint32_t tO = tmem + C::kColO + q * D + lane_off;
      for (int j = 0; j < n_tiles; ++j) {
        const int buf = NQ == 2 ? q : j & 1;
        const uint32_t parity = (NQ == 2 ? j : j >> 1) & 1;
        ok = warp_wait(&mt.s_full[buf], parity, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tS = tmem + buf * 128 + lane_off;
        const int v0 = u0 + j * kT;
        uint32_t vis[4];
        bool full = v0 + kT <= hi_min && (v0 >= lo_max || v0 + kT <= span.sk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vis[i] = mt.valid[j & 7][i];
          full &= vis[i] == 0xFFFFFFFFu;
        }
        if (!full)
#pragma unroll
          for (int i = 0; i < 4; ++i) vis[i] &= sees32(row, span.sk, v0 + 32 * i);
        float mx = full ? row_max<true>(tS, vis) : row_max<false>(tS, vis);
        if (mx > -INFINITY) mx *= c;
        if (__any_sync(0xffffffffu, mx > -INFINITY && !(mx <= m + kChunkTau))) {
          const float n = mx > m + kChunkTau || m == kNoMax ? fmaxf(m, ceilf(mx)) : m;
          const float a = n == m || m == kNoMax ? 1.f : exp2_int(m - n);
          m = n;
          l *= a;
          if (j > 0 && __any_sync(0xffffffffu, a != 1.f)) {
            // O holds the PVs of the tiles before this one.  Two row tiles: S(j)
            // was issued behind PV(j-1), so s_full covers it; one: s_full
            // covers PV(j-2), and this waits for PV(j-1).
            bool go = true;
            if (NQ == 1) go = warp_wait(&mt.o_done, (j - 1) & 1, abort_flag);
            tc_fence_after();
            if (go) {
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 16) {
                uint32_t o[16];
                tmem_ld16(tO + c0, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                tmem_st16(tO + c0, o);
              }
            }
          }
        }
        const float sh = kChunkPShift - (m == kNoMax ? 0.f : m);
        l += full ? exp_tile<true>(tS, vis, c, sh) : exp_tile<false>(tS, vis, c, sh);
        tc_fence_before();
        mbar_arrive(&mt.p_ready[buf]);
      }
      // ====================================================== epilogue
      if (ok) ok = warp_wait(&mt.o_all[q], 0, abort_flag);
      tc_fence_after();
      if (ok) {
        const bool live = rr < RC;
        const float vs = p.v_scale_dev ? *p.v_scale_dev : p.v_scale;
        const int64_t vec = live ? vec_of(rr) : 0;
        const bool dead = l == 0.f;
        const float f = p.S > 1 ? kChunkInvPShift : (dead ? 0.f : vs / l);
        const int pr = work.row0 + rr;
        uint16_t* dst = p.out + (int64_t)(req.row0 + pr / p.G) * p.o_st + (int64_t)(g * p.G + pr % p.G) * p.o_sh;
        if (p.S > 1 && live) p.ml[s * plane + vec] = make_float2(m, l * kChunkInvPShift);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c0, o);
          if (!live) {
          } else if (p.S > 1) {
            float* part = p.partial + (s * plane + vec) * D + c0;
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(part + k) =
                  make_float4(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f,
                              __uint_as_float(o[k + 2]) * f, __uint_as_float(o[k + 3]) * f);
          } else {
            uint32_t y[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2)
              y[k / 2] = dead ? 0u : pack_out<DT>(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f);
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<uint4*>(dst + c0 + 2 * k) = make_uint4(y[k], y[k + 1], y[k + 2], y[k + 3]);
          }
          __syncwarp();
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ======================================================== decoders
    const int w = warp & 3;
    if constexpr (NQ == 2)
      ok = decode_tiles<D, FMT, true, true>(p, mt, smem, b, g, u0, u1, n_tiles, span, w, lane);
    else if (warp < 8)
      ok = decode_tiles<D, FMT, true, false>(p, mt, smem, b, g, u0, u1, n_tiles, span, w, lane);
    else
      ok = decode_tiles<D, FMT, false, true>(p, mt, smem, b, g, u0, u1, n_tiles, span, w, lane);
  } else {
    // ======================================================== UMMA issue
    // The whole warp walks the schedule and one elected lane issues: operands
    // then stay in uniform registers (issued by a lone diverged lane, each UMMA cost
    // its thread ~80 cycles, more than the 65 that the tensor core needs).
    constexpr int NS = C::kStages;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t idesc_qk = idesc_f16_f32(kM, kT, false, false);
    const uint32_t idesc_pv = idesc_f16_f32(kM, D, false, true);
    const uint64_t qdesc = smem_desc(smem_u32(smem + C::kOffQ), 16, 1024, kSw128);
    const uint64_t kdesc = smem_desc(smem_u32(smem + C::kOffK), 16, 1024, kSw128);
    const uint64_t vdesc = smem_desc(smem_u32(smem + C::kOffV), kT * 128, 1024, kSw128);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && warp_wait(bar, parity, abort_flag);
      tc_fence_after();
      return ok;
    };
    static_assert(kM == kT, "Q and K tiles share their block stride");
    // S(buf) = Q_q . K_j^T, then the barriers that it completes
    auto qk = [&](int q, int buf, int j, bool k_last) {
      const uint64_t qd = qdesc + (uint64_t)((q * (kM * D * 2)) >> 4);
      const uint64_t kd = kdesc + (uint64_t)(((j % NS) * C::kOpBytes) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t step = (uint64_t)(((kk / 4) * (kM * 128) + (kk % 4) * 32) >> 4);
          mma_ss(tm + buf * 128, qd + step, kd + step, idesc_qk, kk > 0);
        }
        mma_commit(&mt.s_full[buf]);
        if (k_last) mma_commit(&mt.k_empty[j % NS]);
      }
    };
    // O_q += P(buf) . V_j
    auto pv = [&](int q, int buf, int j, bool v_last, uint64_t* done) {
      const uint64_t vd = vdesc + (uint64_t)(((j % NS) * C::kOpBytes) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kT / 16; ++kk)
          mma_ts(tm + C::kColO + q * D, tm + buf * 128 + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_pv,
                 (j > 0 || kk > 0) ? 1u : 0u);
        if (v_last) mma_commit(&mt.v_empty[j % NS]);
        if (done) mma_commit(done);
      }
    };
    if (wait(&mt.q_full, 0) && wait(&mt.k_full[0], 0)) {
      if (NQ == 2) {
        // S and P of a row tile share their columns: QK(j+1) follows PV(j) in
        // issue order, in which the tensor core runs one CTA's UMMAs
        for (int q = 0; q < nq; ++q) qk(q, q, 0, q == nq - 1);
        for (int j = 0; j < n_tiles && ok; ++j) {
          if (!wait(&mt.v_full[j % NS], (j / NS) & 1)) break;
          for (int q = 0; q < nq; ++q) {
            if (!wait(&mt.p_ready[q], j & 1)) break;
            pv(q, q, j, q == nq - 1, j + 1 == n_tiles ? &mt.o_all[q] : nullptr);
            if (j + 1 == n_tiles) continue;
            if (q == 0 && !wait(&mt.k_full[(j + 1) % NS], ((j + 1) / NS) & 1)) break;
            qk(q, q, j + 1, q == nq - 1);
          }
        }
      } else {
        qk(0, 0, 0, true);
        for (int j = 0; j < n_tiles; ++j) {
          if (j + 1 < n_tiles) {
            // its buffer held P(j-1), whose PV was issued before
            if (!wait(&mt.k_full[(j + 1) % NS], ((j + 1) / NS) & 1)) break;
            qk(0, (j + 1) & 1, j + 1, true);
          }
          if (!wait(&mt.v_full[j % NS], (j / NS) & 1) || !wait(&mt.p_ready[j & 1], (j >> 1) & 1)) break;
          pv(0, j & 1, j, true, j + 1 == n_tiles ? &mt.o_all[0] : &mt.o_done);
        }
      }
    }
    // every UMMA issued must be done before TMEM is freed
    if (elect_one()) mma_commit(&mt.drain);
    __syncwarp();
    mbar_wait_plain(&mt.drain, 0, kPolls);
  }
  if (!ok) set_status(p.status, FP8KV_STATUS_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (mt.vbad) {
    // non-finite V codes (entered as 0): the elements of the rows that see them
    uint32_t* kinds = reinterpret_cast<uint32_t*>(smem + C::kOffQ);
    static_assert(ROWS * D <= C::kOffMeta, "room for the marks");
    mark_nonfinite_v<D, FMT>(p, kinds, b, g, u0, u1, span, RC,
                             [&](int i) { return chunk_row(p, req, span, (work.row0 + i) / p.G); });
    const float vs = p.v_scale_dev ? *p.v_scale_dev : p.v_scale;
    for (int x = tid; x < RC * D; x += kTileThreads) {
      const int i = x / D, d = x % D;
      const uint32_t kind = (kinds[i * (D / 4) + d / 4] >> (8 * (d % 4))) & 0xFFu;
      if (!kind) continue;
      const float v = nonfinite_value(kind);
      if (p.S > 1) {
        p.partial[(s * plane + vec_of(i)) * D + d] = v;
      } else {
        const int rr = work.row0 + i;
        p.out[(int64_t)(req.row0 + rr / p.G) * p.o_st + (int64_t)(g * p.G + rr % p.G) * p.o_sh + d] =
            (uint16_t)(pack_out<DT>(v * vs, 0.f) & 0xFFFFu);
      }
    }
  }
}

template <int D, int FMT, int DT>
cudaError_t run(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  auto fn = chunk_tile<D, FMT, DT>;
  constexpr int smem = TileCfg<D>::kSmem;
  static DeviceOnce once;
  cudaError_t e = once.run([&] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  fn<<<dim3(p.row_tiles, p.Hkv, p.S), kTileThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t pick(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  constexpr int E4 = FP8KV_KV_E4M3, E5 = FP8KV_KV_E5M2, F16 = FP8KV_DTYPE_F16, BF16 = FP8KV_DTYPE_BF16;
  if (plan->kv_format == E5)
    return plan->dtype == BF16 ? run<D, E5, BF16>(plan, p, st) : run<D, E5, F16>(plan, p, st);
  return plan->dtype == BF16 ? run<D, E4, BF16>(plan, p, st) : run<D, E4, F16>(plan, p, st);
}

}  // namespace

cudaError_t launch_chunk_tile(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  switch (plan->head_dim) {
    case 64: return pick<64>(plan, p, st);
    case 128: return pick<128>(plan, p, st);
    default: return pick<256>(plan, p, st);
  }
}

}  // namespace fp8kv
