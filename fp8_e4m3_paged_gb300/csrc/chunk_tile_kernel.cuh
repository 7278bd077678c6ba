#pragma once

// Chunk attention for many query vectors: tcgen05 tiles of 128 vectors by 128
// positions.
//
// The query heads of one KV head and the new tokens of one request are packed
// into rows (token * G + head), so a tile is full whatever the group size and
// one decode of K and V serves all of them.  A CTA owns 256 rows (two row
// tiles; 128 rows for D = 256) of one request and KV head, and one partition
// of the positions that its rows see.  Twelve warps, so that each thread may
// have 168 registers (a row of S is 128 of them):
//   warps 0-3, 4-7   row tiles 0 and 1 (thread = row = TMEM lane): softmax, and
//                    the first warp of the four issues the row tile's UMMAs;
//                    D = 256: warps 0-3 only, and warps 4-7 decode K;
//   warps 8-11       decode K and V (D = 256: V): FP8 rows, requested one tile
//                    ahead into registers, to swizzled fp16 operand tiles.
// Per tile j and row tile q:  S_q = Q_q . K_j^T (M 128, N 128),
// P_q = 2^(s - m + 7) as fp16 over S_q in TMEM, O_q += P_q . V_j (A from TMEM).
// Two row tiles alternate: while one's softmax runs, the tensor core works on
// the other's PV(j) and QK(j+1), issued together.  For D = 256 two S buffers of the
// one row tile do the same: QK of tile j+1 is issued between the halves (64
// positions each) of PV(j).
//
// What bounds it: the four phases of a tile (decode, QK, softmax, PV) share an
// SM's issue slots and shared memory.  Per tile of 256 x 128 (D 128) the UMMAs take
// 2048 cycles; the exponentials, the conversions and the decode about 2000 issue
// cycles per scheduler, and operand reads, decode stores and Q/P traffic 2300
// shared-memory cycles; together they run in 3400 to 3600.  32 heads over 8, D 128,
// 2048 queries on 30000 cached positions: 865 us, 1204 TFLOP/s (the FP16 dense rate
// would take 537); 8192 queries with window 1024: 177 us, of which a CTA's
// start and end (about 12 us: lengths, Q, the first rows, the output) are the
// larger part of what lies above the tensor time.
// Measured and not taken: 16 warps of 128 registers with K and V decoded by four
// warps each (984 us where this took 955), the same split by setmaxnreg (1076 and
// more), row tiles in strict turns (955 to 978), a running maximum one tile late
// (986), and one persistent CTA per SM with equal shares of all tiles (890 for
// the long prompt, but 220 for the windowed one and 236 for 16 requests: the
// pieces' changes cost more than the gaps that they fill).
// TMEM: S at columns 0 and 128, O at 256 (256 columns).
//
// Every wait is bounded (see split_tc_kernel.cuh): a wait that gives up sets the
// CTA's abort flag and FP8KV_STATUS_TIMEOUT, every role stops, and the issued
// UMMAs are drained before TMEM is freed.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk_common.cuh"
#include "chunk_schedule.h"
#include "dependent.cuh"
#include "internal.h"
#include "tc_ptx.cuh"
#include "tile_rows.cuh"

namespace fp8kv {
namespace {

using namespace tc;

constexpr int kTileThreads = 12 * 32;
constexpr int kStagesMax = 4;
constexpr int kMetaBytes = 4096;

template <int D>
struct TileCfg : RowCfg<D> {
  static constexpr int kNQ = D == 256 ? 1 : 2;
  static constexpr int kStages = D == 256 ? 1 : D == 128 ? 2 : 4;  // K stages, and V stages
  // V's barriers: one per stage; D = 256: one per half (64 positions) of the only stage,
  // which is decoded anew as soon as PV of that half is done.  (With one for the
  // whole tile, PV of the next tile waited for 2500 cycles of decode behind PV of this
  // one: 87 us for 1000 queries of 6 heads on 8192 positions, 82 so; 84 with the care for
  // large logits and NaN since.)
  static constexpr int kVStages = D == 256 ? 2 : kStages;
  static constexpr int kOpBytes = kT * D * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kNQ * kM * D * 2;
  static constexpr int kOffV = kOffK + kStages * kOpBytes;
  static constexpr int kOffMeta = kOffV + kStages * kOpBytes;
  static constexpr int kSmem = kOffMeta + kMetaBytes + 1024;  // meta, alignment
  static constexpr uint32_t kColO = 256;
  static_assert(kNQ * D <= 256 && kSmem <= 232448, "TMEM and shared memory");
};

struct TileMeta {
  uint64_t q_full[2], drain[2];
  uint64_t k_full[kStagesMax], k_empty[kStagesMax], v_full[kStagesMax], v_empty[kStagesMax];
  uint64_t s_full[2], o_all[2];                 // o_all: a row tile's last PV is done
  uint64_t p_ready[2][2];                       // P by halves (p_ready_at)
  uint64_t o_done;                              // D = 256: PV(j) is done, every tile but the last
  alignas(16) uint32_t valid[8][4];             // per tile (j % 8): positions whose block is in range
  int64_t place[2][4][32];                      // per decoder warp: byte offsets of its rows
  float sum[256];                               // the rows' sums, for non-finite V codes
  uint32_t tmem, abort, vbad;
};
static_assert(sizeof(TileMeta) <= kMetaBytes, "meta block");

// V pieces before they are stored: zero for rows whose block is out of range or that
// lie past the partition (their weight is 0, and 0 * NaN would not be; K rows
// need not, their logits are masked), and non-finite codes as zero (returns
// true if there were any).
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
  constexpr int NS = C::kStages;
  volatile uint32_t* const abort_flag = &mt.abort;
  const uint8_t* kbase = p.k_cache + g * p.ksh;
  const uint8_t* vbase = p.v_cache + g * p.vsh;
  // Position 32 w + lane of a tile: its block id is requested one tile before
  // the place is needed, so that nothing waits for that load either.  From
  // tile to tile page and slot move by a constant step.
  const int32_t* table = p.block_table + (int64_t)b * p.bt_stride;
  const int step_page = kT / p.page_size, step_slot = kT - step_page * p.page_size;
  int v_ask = u0 + 32 * w + lane, page = 0, slot = 0;
  auto locate_token = [&]() {
    const int pos = span.position(v_ask);
    page = div_page(pos, p.page_size, p.page_div);
    slot = pos - page * p.page_size;
  };
  locate_token();
  int blk = -1, slot_now = 0;
  bool in = false;
  auto ask = [&]() {  // of the next tile in order
    in = v_ask < u1;
    blk = -1;
    slot_now = slot;
    if (in) blk = __ldg(table + page);
    const bool sink = v_ask < span.sk;
    v_ask += kT;
    page += step_page;
    slot += step_slot;
    if (slot >= p.page_size) {
      slot -= p.page_size;
      ++page;
    }
    if (sink) locate_token();  // the window may begin in between
  };
  const bool same = p.ksb == p.vsb && p.kst == p.vst;  // K and V rows at the same offset
  int64_t koff = 0, voff = 0;
  uint32_t ok_next = 0u;
  auto find = [&]() {
    const bool ok = blk >= 0 && blk < p.num_kv_blocks;
    if (DO_K && in && !ok) set_status(p.status, FP8KV_STATUS_BAD_BLOCK);
    if (DO_K) koff = ok ? blk * p.ksb + (int64_t)slot_now * p.kst : 0;
    if (DO_V) voff = DO_K && same ? koff : ok ? blk * p.vsb + (int64_t)slot_now * p.vst : 0;
    ok_next = __ballot_sync(0xffffffffu, ok);
  };
  int64_t* place = mt.place[DO_K ? 0 : 1][w];
  uint4 kr[DO_K ? C::kIts : 1], vr[DO_V ? C::kIts : 1];
  auto fetch_k = [&]() {
    __syncwarp();
    place[lane] = koff;
    __syncwarp();
    if constexpr (DO_K) fetch_rows<D>(kbase, place, lane, kr);
  };
  auto fetch_v = [&]() {
    if (!DO_K || !same) {
      __syncwarp();
      place[lane] = voff;
      __syncwarp();
    }
    if constexpr (DO_V) fetch_rows<D>(vbase, place, lane, vr);
  };
  ask();
  find();
  if (DO_K) fetch_k();
  if (DO_V) fetch_v();
  uint32_t ok_now = ok_next;
  ask();
  bool ok = true, bad = false;
  for (int j = 0; j < n_tiles; ++j) {
    const int st = j % NS;
    const uint32_t empty_parity = ((j / NS) - 1) & 1;
    if (j + 1 < n_tiles) {
      find();
      ask();
    }
    // (the last tile is requested again: the requests stay unconditional)
    if constexpr (DO_K) {
      if (j >= NS && !warp_wait(&mt.k_empty[st], empty_parity, abort_flag)) {
        ok = false;
        break;
      }
      store_rows<D, FMT>(smem + C::kOffK + st * C::kOpBytes, kr, 32 * w, lane);
      // K(j+8) is decoded after QK(j+4) at the earliest, and that after softmax j+3
      if (lane == 0) mt.valid[j & 7][w] = ok_now;
      fence_proxy_async_smem();
      mbar_arrive(&mt.k_full[st]);
      fetch_k();
    }
    if constexpr (DO_V) {
      bad |= clean_v<D, FMT>(vr, ok_now, lane);
      const int vs = C::kNQ == 1 ? w / 2 : st;
      if (j >= NS && !warp_wait(&mt.v_empty[vs], empty_parity, abort_flag)) {
        ok = false;
        break;
      }
      store_rows<D, FMT>(smem + C::kOffV + st * C::kOpBytes, vr, 32 * w, lane);
      fence_proxy_async_smem();
      mbar_arrive(&mt.v_full[vs]);
      fetch_v();
    }
    ok_now = ok_next;
  }
  if (bad) mt.vbad = 1u;
  return ok;
}

// P = 2^(c S + sh) as fp16 for 64 of a row's logits; adds to the row's sums.
__device__ __forceinline__ void exp_half(const uint32_t* x, uint64_t c2, uint64_t sh2, uint64_t (&sum)[2],
                                         uint32_t (&y)[32]) {
#pragma unroll
  for (int k = 0; k < 64; k += 2) {
    const float2 e = unpair(fma2(pair(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), c2, sh2));
    const float p0 = fast_exp2(e.x), p1 = fast_exp2(e.y);
    sum[(k / 2) & 1] = add2(sum[(k / 2) & 1], pair(p0, p1));
    y[k / 2] = pack_half2(p0, p1);
  }
}

// TREE: new tokens see each other by their masks.
template <int D, int FMT, int DT, bool TREE>
__global__ void __launch_bounds__(kTileThreads, 1) chunk_tile(const __grid_constant__ ChunkParams p) {
  using C = TileCfg<D>;
  constexpr int NQ = C::kNQ, ROWS = NQ * kM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TileMeta& mt = *reinterpret_cast<TileMeta*>(smem + C::kOffMeta);
  const int tid = threadIdx.x, lane = tid & 31;
  // (broadcast: known to be the same in all lanes, so that branches are uniform and a
  // UMMA's operands stay in uniform registers: 955 us became 922)
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (TREE) let_next_kernel_start();
  const int g = blockIdx.x % p.Hkv, tile = blockIdx.x / p.Hkv;
  int s = blockIdx.y, share_len = 0;

  TileWork work;
  if (TREE && p.per_head > 0) {
    Share share;
    const bool found = share_of<true>(p, p.per_head, tile, lane, share);
    // (the join derives every request's partitions from the length for requests of two row tiles)
    if (blockIdx.x == 0 && tid == 0) *p.share = share.base;
    if (!found) return;
    work = {share.b, 0};
    s = share.s;
    share_len = share.T * kT;
  } else if (!locate(p, ROWS, tile, lane, work)) {
    return;
  }
  const int b = work.b;
  const ChunkRequest req = chunk_request(p, b);
  const int RC = min(ROWS, req.n * p.G - work.row0);
  if (RC <= 0 || work.row0 < 0) return;
  const int64_t plane = (int64_t)p.total_q * p.Hq;
  auto vec_of = [&](int r) {
    const int rr = work.row0 + r;
    return (int64_t)(req.row0 + rr / p.G) * p.Hq + g * p.G + rr % p.G;
  };
  const ChunkSpan span = chunk_span<TREE>(p, req, work.row0 / p.G, (work.row0 + RC - 1) / p.G);
  int per = min((span.U + p.parts - 1) / p.parts, p.max_part);
  per = (per + kT - 1) / kT * kT;
  if (TREE && p.per_head > 0) per = share_len;
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
  const int nq = __shfl_sync(0xffffffffu, NQ == 2 && RC > kM ? 2 : 1, 0);  // row tiles in use

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&mt.k_full[i], 128);
      mbar_init(&mt.k_empty[i], nq);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&mt.v_full[i], NQ == 1 ? 64 : 128);
      mbar_init(&mt.v_empty[i], nq);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&mt.q_full[i], kM);
      mbar_init(&mt.drain[i], 1);
      mbar_init(&mt.s_full[i], 1);
      mbar_init(&mt.p_ready[i][0], 4);  // one lane of each of the row tile's warps
      mbar_init(&mt.p_ready[i][1], 4);
      mbar_init(&mt.o_all[i], 1);
    }
    mbar_init(&mt.o_done, 1);
    mt.abort = 0u;
    mt.vbad = 0u;
    mbar_init_fence();
  }
  if (warp == 0) {
    tmem_alloc(&mt.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, mt.tmem, 0);
  volatile uint32_t* const abort_flag = &mt.abort;
  const float ks = p.k_scale_dev ? *p.k_scale_dev : p.k_scale;
  const float cf = p.softmax_scale * ks * kLog2e;  // base-2 logit factor
  bool ok = true;

  if (warp < 4 * NQ) {
    const int q = warp >> 2;
    if (q < nq) {
      // ====================================================== Q tile
      // One warp per row: fp16 as it is, bf16 scaled by a power of two; the
      // sign of the logit factor goes into Q.
      constexpr int V = D / 32;  // elements per lane
      constexpr int kRowsAtOnce = D == 256 ? 16 : 32;  // 64 registers
      uint8_t* sQ = smem + C::kOffQ + q * (kM * D * 2);
      const uint32_t flip = cf < 0.f ? 0x80008000u : 0u;
      const int e = lane * V;  // first element of the lane
      float back = 1.f;        // inverse scale of this thread's row
      // the warp's first row; rows past RC read the last one (their results are dropped)
      int rr0 = min(q * kM + 32 * (warp & 3), RC - 1);
      int head = (work.row0 + rr0) % p.G;
      const uint16_t* src =
          p.q + (int64_t)(req.row0 + (work.row0 + rr0) / p.G) * p.q_st + (int64_t)(g * p.G + head) * p.q_sh + e;
#pragma unroll 1
      for (int k0 = 0; k0 < 32; k0 += kRowsAtOnce) {
        uint32_t w[kRowsAtOnce][V / 2];
        // all loads first
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k) {
          if constexpr (V == 2) {
            w[k][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
          } else if constexpr (V == 4) {
            *reinterpret_cast<uint2*>(w[k]) = __ldg(reinterpret_cast<const uint2*>(src));
          } else {
            *reinterpret_cast<uint4*>(w[k]) = __ldg(reinterpret_cast<const uint4*>(src));
          }
          if (++rr0 < RC) {
            const bool wrap = ++head == p.G;
            if (wrap) head = 0;
            src += wrap ? p.q_st - (p.G - 1) * p.q_sh : p.q_sh;
          }
        }
        // bf16: all rows' maxima at once, then each lane the scale of one row.  The maxima
        // (as integers: a NaN is larger than every number, and is not dropped) go
        // through a butterfly that halves the rows a lane holds in each step, two rows
        // to a register: 16 shuffles for 32 rows, where 32 warp reductions took 2000
        // cycles more of a CTA's start.
        RowScale own = {1.f, 1.f};  // of row k0 + lane % kRowsAtOnce
        if (DT == FP8KV_DTYPE_BF16) {
          constexpr int N = kRowsAtOnce;
          auto mag = [&](int k) {
            uint32_t t = w[k][0] & 0x7FFF7FFFu;
#pragma unroll
            for (int i = 1; i < V / 2; ++i) t = __vmaxu2(t, w[k][i] & 0x7FFF7FFFu);
            return t;
          };
          uint32_t t[N / 2];  // rows k and k + N / 2
#pragma unroll
          for (int k = 0; k < N / 2; ++k) {
            const uint32_t a = mag(k), b = mag(k + N / 2);
            t[k] = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
          }
#pragma unroll
          for (int o = N / 4; o >= 1; o /= 2) {
            const bool upper = lane & o;
#pragma unroll
            for (int k = 0; k < o; ++k) {
              const uint32_t give = upper ? t[k] : t[k + o], keep = upper ? t[k + o] : t[k];
              t[k] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, give, o));
            }
          }
#pragma unroll
          for (int o = N / 2; o < 32; o *= 2) t[0] = __vmaxu2(t[0], __shfl_xor_sync(0xffffffffu, t[0], o));
          own = row_scale_bf16(__uint_as_float(lane & (N / 2) ? t[0] & 0xFFFF0000u : t[0] << 16));
          if (lane / N == k0 / N) back = own.back;
          if (flip) own.to_f16 = -own.to_f16;
        }
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k) {
          const int r = 32 * (warp & 3) + k0 + k;
          if (DT == FP8KV_DTYPE_BF16) {
            const float to_f16 = __shfl_sync(0xffffffffu, own.to_f16, k);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              const float2 x = unpair(mul2(pair(__uint_as_float(w[k][i] << 16), __uint_as_float(w[k][i] & 0xFFFF0000u)),
                                           pair(to_f16, to_f16)));
              w[k][i] = pack_half2(x.x, x.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[k][i] ^= flip;
          }
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
      mbar_arrive(&mt.q_full[q]);

      // ====================================================== UMMA issue
      // The row tile's first warp walks the schedule and one elected lane issues
      // (operands of a converged warp stay in uniform registers).  S and P of
      // a row tile share their columns: QK(j+1) follows PV(j) in issue order, in
      // which the tensor core runs one thread's UMMAs.
      const bool issuer = (warp & 3) == 0;
      constexpr int NS = C::kStages;
      static_assert(kM == kT, "Q and K tiles share their block stride");
      const uint32_t idesc_qk = idesc_f16_f32(kM, kT, false, false);
      const uint32_t idesc_pv = idesc_f16_f32(kM, D, false, true);
      const uint64_t qdesc = smem_desc(smem_u32(smem + C::kOffQ + q * (kM * D * 2)), 16, 1024, kSw128);
      const uint64_t kdesc = smem_desc(smem_u32(smem + C::kOffK), 16, 1024, kSw128);
      const uint64_t vdesc = smem_desc(smem_u32(smem + C::kOffV), kT * 128, 1024, kSw128);
      auto buf_of = [&](int j) { return NQ == 2 ? q : j & 1; };
      auto issue_qk = [&](int j) {
        ok = ok && warp_wait(&mt.k_full[j % NS], (j / NS) & 1, abort_flag);
        if (!ok) return;
        tc_fence_after();
        const uint64_t kd = kdesc + (uint64_t)(((j % NS) * C::kOpBytes) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t step = (uint64_t)(((kk / 4) * (kM * 128) + (kk % 4) * 32) >> 4);
            mma_ss(tmem + buf_of(j) * 128, qdesc + step, kd + step, idesc_qk, kk > 0);
          }
          mma_commit(&mt.s_full[buf_of(j)]);
          mma_commit(&mt.k_empty[j % NS]);
        }
      };
      // PV of half h, once every warp has written its rows of P
      auto issue_pv = [&](int j, int h) {
        const int vs = NQ == 1 ? h : j % NS;
        if (NQ == 1 || h == 0) ok = ok && warp_wait(&mt.v_full[vs], (j / NS) & 1, abort_flag);
        const BarrierAt pr = p_ready_at(NQ, q, h, j);
        ok = ok && warp_wait(&mt.p_ready[pr.slot][h], pr.parity, abort_flag);
        if (!ok) return;
        tc_fence_after();
        const uint64_t vd = vdesc + (uint64_t)(((j % NS) * C::kOpBytes) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kT / 32; ++k) {
            const int kk = h * (kT / 32) + k;
            mma_ts(tmem + C::kColO + q * D, tmem + buf_of(j) * 128 + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4),
                   idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
          }
          if (NQ == 1 || h == 1) mma_commit(&mt.v_empty[vs]);
          if (h == 1) {
            if (j + 1 == n_tiles)
              mma_commit(&mt.o_all[q]);
            else if (NQ == 1)
              mma_commit(&mt.o_done);
          }
        }
      };
      if (issuer) {
        ok = warp_wait(&mt.q_full[q], 0, abort_flag);
        issue_qk(0);
      }

      // ====================================================== softmax
      const int rr = q * kM + 32 * (warp & 3) + lane;  // this thread's row of the CTA
      const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
      // (not 0, so that c * -inf stays -inf for masked logits; nor NaN, for the same reason: a
      // NaN scale goes into the rows' sums at the end)
      const float c = fmaxf(fabsf(cf) * back, 1e-30f);
      auto row = any_row<TREE>(0);  // rows past RC: everything, dropped at the end
      if (rr < RC) row = chunk_row<TREE>(p, req, span, (work.row0 + rr) / p.G);
      const int hi_min = __reduce_min_sync(0xffffffffu, row.hi), lo_max = __reduce_max_sync(0xffffffffu, row.lo);
      float m = kNoMax, l = 0.f;
      bool far = false;  // some row of the warp has logits past 2^22
      const uint32_t tO = tmem + C::kColO + q * D + lane_off;
      for (int j = 0; j < n_tiles; ++j) {
        const int buf = buf_of(j);
        ok = ok && warp_wait(&mt.s_full[buf], (NQ == 2 ? j : j >> 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tS = tmem + buf * 128 + lane_off;
        const int v0 = u0 + j * kT;
        const uint4 there = *reinterpret_cast<const uint4*>(mt.valid[j & 7]);
        uint32_t x[128];
        tmem_ld128(tS, x);
        if ((there.x & there.y & there.z & there.w) != 0xFFFFFFFFu || v0 + kT > hi_min ||
            !(v0 >= lo_max || v0 + kT <= span.sk)) {
          // logits that the row does not see become -inf (a NaN among them too)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t vis = i == 0 ? there.x : i == 1 ? there.y : i == 2 ? there.z : there.w;
            if constexpr (TREE)
              vis &= sees32(row, span.sk, v0 + 32 * i, (req.n + 31) / 32);
            else
              vis &= sees32(row, span.sk, v0 + 32 * i);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[32 * i + k] = ((vis >> k) & 1u) ? x[32 * i + k] : 0xFF800000u;
          }
        }
        // row maximum (a NaN is passed over: it makes the sum NaN)
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(x[k + 2 * i])), __uint_as_float(x[k + 2 * i + 1]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        if (__any_sync(0xffffffffu, top - m > kChunkTau)) {  // (false where both are -inf)
          const float n = top - m > kChunkTau ? fmaxf(m, ceilf(top)) : m;
          const float a = n == m || m == kNoMax ? 1.f : exp2_whole(m - n);
          m = n;
          far = __any_sync(0xffffffffu, fabsf(m) >= 0x1p22f && m != kNoMax);
          l *= a;
          if (j > 0 && __any_sync(0xffffffffu, a != 1.f)) {
            // O holds the PVs of the tiles before this one.  Two row tiles: S(j)
            // was issued behind PV(j-1), so s_full covers it; one: s_full
            // covers PV(j-2), and this waits for PV(j-1).
            if (NQ == 1) ok = warp_wait(&mt.o_done, (j - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
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
        const float sh = __fadd_rd(kChunkPShift, m == kNoMax ? -0.f : -m);
        if (far) {
          // the maximum is that of the rounded products, which the fma below would not round
#pragma unroll
          for (int k = 0; k < 128; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * c);
        }
        const uint64_t c2 = far ? pair(1.f, 1.f) : pair(c, c), sh2 = pair(sh, sh);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t y[32];
          exp_half(x + 64 * h, c2, sh2, sum, y);
          tmem_st32(tS + 32 * h, y);  // over S, all of which is in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&mt.p_ready[p_ready_at(NQ, q, h, j).slot][h]);
          if (issuer) {
            if (NQ == 1) {
              if (h == 1 && j + 1 < n_tiles) issue_qk(j + 1);  // its buffer held P(j-1)
              issue_pv(j, h);
            } else if (h == 1) {
              // PV(j) and QK(j+1) of a row tile go to the tensor core in one piece: while it
              // runs, the other row tile is at its softmax.  (PV of the first half at
              // h = 0 costs the warp a wait and an issue amid its exponentials.)
              issue_pv(j, 0);
              issue_pv(j, 1);
              if (j + 1 < n_tiles) issue_qk(j + 1);
            }
          }
        }
        const float2 t = unpair(add2(sum[0], sum[1]));
        l += t.x + t.y;
      }
      if (cf != cf && l != 0.f) l = cf;
      if (issuer) {
        // every UMMA issued must be done before TMEM is freed
        if (elect_one()) mma_commit(&mt.drain[q]);
        __syncwarp();
        mbar_wait_plain(&mt.drain[q], 0, kPolls);
        __syncwarp();
      }
      // ====================================================== epilogue
      if (ok) ok = warp_wait(&mt.o_all[q], 0, abort_flag);
      tc_fence_after();
      if (ok) {
        const bool live = rr < RC;
        const float vs = p.v_scale_dev ? *p.v_scale_dev : p.v_scale;
        const int64_t vec = live ? vec_of(rr) : 0;
        const bool dead = l == 0.f, parts = p.S > 1;
        const float f = parts ? kChunkInvPShift : (dead ? 0.f : vs / l);
        if (parts && live) p.ml[s * plane + vec] = make_float2(m, part_sum(l * kChunkInvPShift));
        mt.sum[rr] = l;
        // A thread holds a row, but a store instruction had better write few rows: 128
        // bytes of each of the warp's 32 rows go through shared memory (the
        // warp's part of Q, all reads of which are done; 16-byte chunk c of row r
        // at c ^ (r % 8)) and out as four rows per instruction.  (16 bytes of 32
        // rows each: 5000 to 6000 cycles of a CTA's end.)
        const int pr = work.row0 + rr;
        char* to = nullptr;  // this thread's row
        if (live)
          to = parts ? reinterpret_cast<char*>(p.partial + (s * plane + vec) * D)
                     : reinterpret_cast<char*>(p.out + (int64_t)(req.row0 + pr / p.G) * p.o_st +
                                               (int64_t)(g * p.G + pr % p.G) * p.o_sh);
        char* row_to[8];     // rows 4 i + lane / 8 of the warp
#pragma unroll
        for (int i = 0; i < 8; ++i)
          row_to[i] = reinterpret_cast<char*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), 4 * i + lane / 8));
        uint8_t* buf = smem + C::kOffQ + q * (kM * D * 2) + (warp & 3) * 4096;
        static_assert(kM * D * 2 >= 4 * 4096, "room for the four warps");
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += parts ? 32 : 64) {
          uint4 y[8];
          if (parts) {
            uint32_t o[32];
            tmem_ld32(tO + c0, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          } else {
            uint32_t o[64];
            tmem_ld64(tO + c0, o);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[k] = dead ? 0u : pack_out<DT>(__uint_as_float(o[2 * k]) * f, __uint_as_float(o[2 * k + 1]) * f);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(buf + lane * 128 + ((k ^ (lane & 7)) * 16)) = y[k];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + lane / 8;
            const uint4 v = *reinterpret_cast<const uint4*>(buf + r * 128 + (((lane & 7) ^ (r & 7)) * 16));
            if (row_to[i]) *reinterpret_cast<uint4*>(row_to[i] + c0 * (parts ? 4 : 2) + (lane & 7) * 16) = v;
          }
        }
      }
    }
  } else {
    // ======================================================== decoders
    const int w = warp & 3;
    if constexpr (NQ == 2)
      ok = decode_tiles<D, FMT, true, true>(p, mt, smem, b, g, u0, u1, n_tiles, span, w, lane);
    else if (warp < 8)
      ok = decode_tiles<D, FMT, true, false>(p, mt, smem, b, g, u0, u1, n_tiles, span, w, lane);
    else
      ok = decode_tiles<D, FMT, false, true>(p, mt, smem, b, g, u0, u1, n_tiles, span, w, lane);
  }
  if (!ok) set_status(p.status, FP8KV_STATUS_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (mt.vbad) {
    // non-finite V codes (entered as 0): the elements of the rows that see them
    uint32_t* kinds = reinterpret_cast<uint32_t*>(smem + C::kOffQ);
    static_assert(ROWS * D <= C::kOffMeta, "room for the marks");
    mark_nonfinite_v<D, FMT>(p, kinds, b, g, u0, u1, span, RC,
                             [&](int i) { return chunk_row<TREE>(p, req, span, (work.row0 + i) / p.G); });
    const float vs = p.v_scale_dev ? *p.v_scale_dev : p.v_scale;
    for (int x = tid; x < RC * D; x += kTileThreads) {
      const int i = x / D, d = x % D;
      const uint32_t kind = (kinds[i * (D / 4) + d / 4] >> (8 * (d % 4))) & 0xFFu;
      if (!kind) continue;
      const float v = nonfinite_value(kind);
      if (p.S > 1) {
        p.partial[(s * plane + vec_of(i)) * D + d] = v;
      } else if (mt.sum[i] != 0.f) {
        // over the row's sum, as every other element: an infinity in a row that is NaN
        // for its logits stays NaN
        const int rr = work.row0 + i;
        p.out[(int64_t)(req.row0 + rr / p.G) * p.o_st + (int64_t)(g * p.G + rr % p.G) * p.o_sh + d] =
            (uint16_t)(pack_out<DT>(v * (vs / mt.sum[i]), 0.f) & 0xFFFFu);
      }
    }
  }
}

template <int D, int FMT, int DT, bool TREE>
cudaError_t run(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  auto fn = chunk_tile<D, FMT, DT, TREE>;
  constexpr int smem = TileCfg<D>::kSmem;
  static DeviceOnce once;
  cudaError_t e = once.run([&] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  const dim3 grid = TREE && p.per_head > 0 ? dim3(p.per_head * p.Hkv) : dim3(p.row_tiles * p.Hkv, p.S);
  fn<<<grid, kTileThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <int D, bool TREE>
cudaError_t pick(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  constexpr int E4 = FP8KV_KV_E4M3, E5 = FP8KV_KV_E5M2, F16 = FP8KV_DTYPE_F16, BF16 = FP8KV_DTYPE_BF16;
  if (plan->kv_format == E5)
    return plan->dtype == BF16 ? run<D, E5, BF16, TREE>(plan, p, st) : run<D, E5, F16, TREE>(plan, p, st);
  return plan->dtype == BF16 ? run<D, E4, BF16, TREE>(plan, p, st) : run<D, E4, F16, TREE>(plan, p, st);
}

template <bool TREE>
cudaError_t launch(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  switch (plan->head_dim) {
    case 64: return pick<64, TREE>(plan, p, st);
    case 128: return pick<128, TREE>(plan, p, st);
    default: return pick<256, TREE>(plan, p, st);
  }
}

}  // namespace
}  // namespace fp8kv
