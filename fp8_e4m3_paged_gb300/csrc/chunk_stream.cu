// Chunk attention for few query vectors (at most 16 per CTA: the query heads
// of one KV head times a few new tokens): bound by streaming the cache.
//
// One CTA of four warps per (request, KV head, 16 query vectors, partition);
// each warp walks blocks of 16 virtual tokens (chunk_span) on its own, and the
// four are joined at the end.  A block's rows are requested one to three
// blocks ahead by cp.async into the warp's own ring (whole rows per
// instruction: a copy of half a 128-byte line moves the line), so the loop
// has no CTA barrier.  Each lane then takes the bytes that its MMA fragments hold:
//   S^T[16 tokens x 8 vectors] = K . Q^T, m16n8k16: lane (n = lane/4, c =
//     lane%4) of the A operand needs four d of tokens n and n + 8, so it takes
//     the 16-byte pieces c, c + 4, ... of their rows; a 32-bit word of
//     each decodes to one MMA's A fragment, and the d that the words hold are
//     simply the order in which Q's B fragments are laid out;
//   O^T[16 d x 8 vectors] += V^T . P^T: an A fragment needs two tokens of one
//     d in a register, so the lane takes the same 16-byte piece n of tokens
//     2c, 2c+1, 2c+8, 2c+9 and interleaves their bytes before the decode; P^T's B
//     fragments are S^T's accumulators, packed to fp16 and transposed 8 by 8 (movmatrix),
//     in two halves (twice the vectors' columns, or twice the products).
// Tokens and d as the MMA's 16 rows, vectors as its 8 columns: a decode step's
// 1 to 8 vectors waste no rows, which halves the MMAs and O's registers
// against the other orientation.  Legacy mma.sync rather than tcgen05: with 4 to
// 16 vectors the products are a few percent of the tensor peak, and TMEM or
// shared-memory operands would only add copies and barriers to a kernel whose
// time is the bytes' arrival.  That also pays for P in two fp16 halves.
//
// Partitions of one request and KV head form a thread-block cluster when there
// are at most 8: their sums are joined through distributed shared memory in
// the same launch.  More go through the workspace and chunk_join.
//
// Measured (32 heads over 8, D 128): 57 requests of one token with window 16384,
// every SM with three CTAs: 6.36 TB/s; 64 ragged requests with window 4096, 404 MB:
// 81 us, 5.0 TB/s, because 512 CTAs leave some SMs with four of them and some with
// three.  One request and window 1024: 7.7 us, most of it the launch and the chain
// lengths -> block table -> rows -> join.
#include <algorithm>
#include <climits>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk_common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace fp8kv {
namespace {

constexpr int kWarps = kChunkStreamWarps;
constexpr int kThreadsS = 32 * kWarps;
constexpr int kR = kChunkStreamRows;
constexpr int kBlk = kChunkStreamBlock;
static_assert(kBlk == 16, "an MMA's tokens");

// NQ: columns of 8 query vectors.
template <int D, int NQ>
struct StreamCfg {
  static constexpr int kRows = 8 * NQ;
  static constexpr int kKP = D / 64;                 // 16-byte pieces of a K row per lane
  static constexpr int kVP = D >= 128 ? D / 128 : 1; // pieces of a V row per lane
  static constexpr int kVWords = D >= 128 ? 4 : 2;   // 32-bit words per piece
  static constexpr int kQStride = D + 8;             // fp16 elements (padding: fragment loads without conflicts)
  static constexpr bool kQRegs = D * NQ <= 256;      // Q's fragments stay in registers
  static constexpr int kCtas = D == 256 ? 2 : D == 128 ? (NQ == 1 ? 4 : 3) : (NQ == 1 ? 5 : 4);  // resident per SM
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;  // blocks of a warp in flight or in use
  static constexpr int kCh = D / 16;                 // 16-byte pieces of a row, lanes that copy it
  static constexpr int kRowsIt = 32 / kCh;           // rows that the warp copies at a time
  static constexpr int kRowBytes = kBlk * D;         // a block's K (V) rows
  static constexpr int kRing = kStages * 2 * kRowBytes;  // per warp; then its numerators [row][D]
  static constexpr int kQBytes = kRows * kQStride * 2;
  static constexpr int kOffQ = kWarps * kRing;
  static constexpr int kOffRed = kOffQ + kQBytes;    // per warp: rows' maxima and sums; then inverse row scales
  // Cluster: the joined numerators, as float4 items, are owned by its CTAs in
  // equal runs; an owner receives every partition's items and (maximum, sum) pairs here.
  static constexpr int kItems = kRows * D / 4;
  static constexpr int kIter = (kItems + kThreadsS - 1) / kThreadsS;
  static constexpr int kOffPairs = kOffRed + (2 * kWarps + 1) * 16 * 4;  // [partition][row]
  static constexpr int kOffItems = kOffPairs + kChunkClusterMax * 16 * 8;  // [partition][item of the run]
  static constexpr int kSmem = kOffItems + (kItems + kChunkClusterMax) * 16;
  static_assert(kRing >= kRows * D * 4, "a warp's numerators fit its ring");
  static_assert(kRing * kWarps >= kRows * D, "non-finite marks");
};

// The 8 x 8 matrix of 16-bit elements that the warp holds (row lane/4, columns
// 2 (lane%4) + {0, 1}), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

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

// Thread-block cluster: barrier over all its CTAs in two halves (the first without
// order, for a CTA that has only begun), and stores into a peer's shared memory
// (the place that `p` has in CTA `rank`).
__device__ __forceinline__ void cluster_here() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_store(uint32_t a, float2 x) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(a), "f"(x.x), "f"(x.y) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t a, float4 x) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
               : "memory");
}

__device__ __forceinline__ uint32_t word(const uint4& w, int i) {
  return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// The request with the r-th most positions (at most kThreadsS requests); `key` is room
// for kThreadsS + 1 (a static array would cost the fourth CTA of an SM).
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
    if (rank == r) key[kThreadsS] = t;
  }
  __syncthreads();
  const int b = key[kThreadsS];
  __syncthreads();
  return b;
}

// TWIN (at most 4 vectors): columns 4 to 7 hold the vectors of columns 0 to 3 again.
template <int D, int FMT, int DT, int NQ, bool TWIN>
__global__ void __launch_bounds__(kThreadsS, StreamCfg<D, NQ>::kCtas)
    chunk_stream(const __grid_constant__ ChunkParams p, const int clustered, const int sorted) {
  static_assert(!TWIN || NQ == 1, "one column block");
  using C = StreamCfg<D, NQ>;
  constexpr int ST = C::kStages;
  extern __shared__ __align__(16) uint8_t smem[];
  uint16_t* sQ = reinterpret_cast<uint16_t*>(smem + C::kOffQ);
  float* sML = reinterpret_cast<float*>(smem + C::kOffRed);  // [warp]: 16 maxima, then 16 sums
  float* sBack = sML + 2 * kWarps * 16;                      // [16] inverse row scales

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rq = lane >> 2, c = lane & 3;
  // KV heads next to each other, so that the CTAs that read one token's heads (adjacent
  // in memory) run at the same time; the requests from the longest where there are
  // several CTAs to an SM: the last ones, which only some SMs get, are then short.
  // 64 requests of 512 to 65536 positions in a window of 4096: 80 us so, 90 by index
  // (P in one half then).  Up to as many requests as the CTA has threads; beyond, by index.
  const int nth = div_hkv(p, blockIdx.x), g = blockIdx.x - nth * p.Hkv, s = blockIdx.y;
  const int b = sorted ? by_length(p, reinterpret_cast<int*>(sML), nth) : nth;
  const int row_first = blockIdx.z * kR;  // packed rows: token * G + head of the group
  const ChunkRequest req = chunk_request(p, b);
  if (tid == 0 && req.bad) set_status(p.status, FP8KV_STATUS_BAD_LEN);
  const int RC = min(TWIN ? 4 : kR, req.n * p.G - row_first);
  auto row_of_column = [](int col) { return TWIN ? col & 3 : col; };
  if (RC <= 0) return;  // every CTA of the cluster
  if (clustered) cluster_here();  // peers may write here once all have come this far (ordered: 0.4 us more)
  const int64_t plane = (int64_t)p.total_q * p.Hq;
  auto token_of = [&](int r) { return token_at(p, row_first + r); };
  auto head_of = [&](int r) { return g * p.G + row_at(p, row_first + r).head; };
  auto vec_of = [&](int r) { return (int64_t)(req.row0 + token_of(r)) * p.Hq + head_of(r); };

  const ChunkSpan span = chunk_span(p, req, token_of(0), token_of(RC - 1));
  int per = min(div_parts(p, span.U + p.parts - 1), p.max_part);
  per = (per + kBlk * kWarps - 1) / (kBlk * kWarps) * (kBlk * kWarps);
  const int u0 = (int)min((int64_t)s * per, (int64_t)span.U), u1 = min(span.U, u0 + per);
  if (u0 >= u1 && p.S > 1 && !clustered) {
    if (tid < RC) p.ml[s * plane + vec_of(tid)] = make_float2(kNoMax, 0.f);
    return;
  }

  // Places of a block's tokens, one per lane (both halves of the warp hold
  // them).  The block id is requested a block before it is needed; the copies
  // are unconditional (tokens without a place read the pool's first row and
  // are masked, V also zeroed).
  const uint8_t* kbase = p.k_cache + g * p.ksh + (lane % C::kCh) * 16;
  const uint8_t* vbase = p.v_cache + g * p.vsh + (lane % C::kCh) * 16;
  uint8_t* ring = smem + warp * C::kRing;
  // offsets of a block's rows, where the warp's own maxima and sums go after its
  // loop (a warp that is done must not touch the others' places)
  int64_t* place = reinterpret_cast<int64_t*>(sML + warp * 32);
  static_assert(kBlk * 8 == 32 * 4, "one in place of the other");
  struct Ask {
    int blk, slot;
    bool in;
  };
  auto ask = [&](int t) {
    const int v = t + (lane & (kBlk - 1));
    Ask a = {-1, 0, v < u1};
    if (a.in) {
      const int pos = span.position(v), page = div_page(pos, p.page_size, p.page_div);
      a.slot = pos - page * p.page_size;
      a.blk = __ldg(p.block_table + (int64_t)b * p.bt_stride + page);
    }
    return a;
  };
  // K is read by 2 tokens x 4 pieces at a time, V by 4 even (or odd) tokens x 2
  // pieces (of 8 bytes for D = 64).
  auto k_swz = [](int r) { return D >= 128 ? 4 * (r & 1) : 0; };
  auto v_swz = [](int r) { return D >= 128 ? 2 * ((r >> 1) & 3) : (r >> 1) & 3; };
  // Copies of the block asked for into stage `st`; returns the tokens that are there.
  auto request = [&](const Ask& a, int st) {
    const bool ok = a.blk >= 0 && a.blk < p.num_kv_blocks;
    if (a.in && !ok) set_status(p.status, FP8KV_STATUS_BAD_BLOCK);
    const int64_t koff = ok ? a.blk * p.ksb + (int64_t)a.slot * p.kst : 0;
    const int64_t voff = ok ? a.blk * p.vsb + (int64_t)a.slot * p.vst : 0;
    // 16-byte piece i of row r goes to position i ^ swz(r), so that the reads
    // below find eight different banks
    uint8_t* dst = ring + st * 2 * C::kRowBytes;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      __syncwarp();  // (the first also ends the reads of this stage)
      if (lane < kBlk) place[lane] = kv == 0 ? koff : voff;
      __syncwarp();
#pragma unroll
      for (int it = 0; it < kBlk / C::kRowsIt; ++it) {
        const int r = it * C::kRowsIt + lane / C::kCh, swz = kv == 0 ? k_swz(r) : v_swz(r);
        tc::cp_async16(dst + kv * C::kRowBytes + r * D + (((lane % C::kCh) ^ swz) * 16),
                       (kv == 0 ? kbase : vbase) + place[r]);
      }
    }
    return __ballot_sync(0xffffffffu, ok) & 0xFFFFu;
  };
  constexpr int kStep = kBlk * kWarps;  // a warp's blocks are this far apart
  const int t_first = u0 + kBlk * warp;
  uint32_t there[ST];  // tokens of the blocks in flight, the oldest first
  Ask next;            // the block after them
  auto fill = [&](auto between) {
    Ask first[ST - 1];
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) first[i] = ask(t_first + i * kStep);
    between();
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
      there[i] = t_first + i * kStep < u1 ? request(first[i], i) : 0u;
      cp_commit();
    }
    next = ask(t_first + (ST - 1) * kStep);
  };

  // Q -> shared memory as fp16 (bf16 rows scaled by a power of two); rows past
  // RC are zero.  One warp per row; the rows are requested before the first
  // blocks, so that their latencies overlap.
  constexpr int V = D / 32;  // elements per lane
  constexpr int kQRows = C::kRows / kWarps;
  uint32_t qw[kQRows][V / 2];
  const float ks = p.k_scale_dev ? __ldg(p.k_scale_dev) : p.k_scale;
  const float vs = p.v_scale_dev ? __ldg(p.v_scale_dev) : p.v_scale;
  fill([&]() {
#pragma unroll
    for (int k = 0; k < kQRows; ++k) {
      const int r = min(row_of_column(warp + k * kWarps), RC - 1);
      const uint16_t* src = p.q + (int64_t)(req.row0 + token_of(r)) * p.q_st + (int64_t)head_of(r) * p.q_sh;
      if constexpr (V == 2)
        qw[k][0] = __ldg(reinterpret_cast<const uint32_t*>(src) + lane);
      else if constexpr (V == 4)
        *reinterpret_cast<uint2*>(qw[k]) = __ldg(reinterpret_cast<const uint2*>(src) + lane);
      else
        *reinterpret_cast<uint4*>(qw[k]) = __ldg(reinterpret_cast<const uint4*>(src) + lane);
    }
  });
  const float cf = p.softmax_scale * ks * kLog2e;
  const uint32_t flip = cf < 0.f ? 0x80008000u : 0u;  // logit factors are non-negative from here on
#pragma unroll
  for (int k = 0; k < kQRows; ++k) {
    const int r = warp + k * kWarps;
    uint32_t* w = qw[k];
    float back = 1.f;
    if (DT == FP8KV_DTYPE_BF16) {
      uint32_t top = 0u;  // as integers: a NaN is larger than every number, and is not dropped
#pragma unroll
      for (int j = 0; j < V / 2; ++j) top = max(top, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
      const RowScale rs = row_scale_bf16(__uint_as_float(__reduce_max_sync(0xffffffffu, top)));
#pragma unroll
      for (int j = 0; j < V / 2; ++j)
        w[j] = pack_half2(__uint_as_float(w[j] << 16) * rs.to_f16, __uint_as_float(w[j] & 0xFFFF0000u) * rs.to_f16);
      back = rs.back;
    }
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
      *reinterpret_cast<uint32_t*>(sQ + r * C::kQStride + lane * V + 2 * j) = row_of_column(r) < RC ? w[j] ^ flip : 0u;
    if (lane == 0) sBack[r] = back;
  }
  __syncthreads();

  // This lane's query vectors 8 n + 2 c + e: logit factors and what they see;
  // vectors past RC see everything (their values are dropped).
  float cq[NQ][2];
  ChunkRow row[NQ][2];
  int hi_min = INT_MAX, lo_max = INT_MIN;
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * c + e;
      cq[n][e] = fabsf(cf) * sBack[r];
      row[n][e] = {INT_MAX, INT_MIN};
      if (row_of_column(r) < RC) row[n][e] = chunk_row(p, req, span, token_of(row_of_column(r)));
      hi_min = min(hi_min, row[n][e].hi);
      lo_max = max(lo_max, row[n][e].lo);
    }
  hi_min = __reduce_min_sync(0xffffffffu, hi_min);
  lo_max = __reduce_max_sync(0xffffffffu, lo_max);

  // Q's B fragments: step (i, w) covers d = 16 (c + 4 i) + 4 w + {0..3} of lane c
  auto q_frag = [&](int n, int i, int w) {
    return *reinterpret_cast<const uint2*>(sQ + (8 * n + rq) * C::kQStride + (c + 4 * i) * 16 + 4 * w);
  };
  uint2 qb[NQ][C::kQRegs ? D / 16 : 1];
  if (C::kQRegs) {
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int i = 0; i < C::kKP; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) qb[n][C::kQRegs ? i * 4 + w : 0] = q_frag(n, i, w);
  }

  float o[D / 16][NQ][4];         // O^T: d tiles of 16
  float m[NQ][2], l[NQ][2];       // running maxima (whole numbers, base 2); sums over this lane's tokens
  float4 acc[C::kIter];           // after the join: numerators of this thread's items, their rows' maxima and sums
  float Ms[C::kIter], Ls[C::kIter];
  bool zap = false;               // second pass: non-finite V codes enter as 0
  while (true) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
      m[n][0] = m[n][1] = kNoMax;
      l[n][0] = l[n][1] = 0.f;
    }
    int st = 0;
    for (int t = t_first; t < u1; t += kStep) {
      // the block ST - 1 ahead goes where the block before this one was
      there[ST - 1] = 0u;
      if (t + (ST - 1) * kStep < u1) {
        there[ST - 1] = request(next, st == 0 ? ST - 1 : st - 1);
        next = ask(t + ST * kStep);
      }
      cp_commit();
      cp_wait<ST - 1>();
      __syncwarp();
      const uint8_t* krows = ring + st * 2 * C::kRowBytes;
      const uint8_t* vrows = krows + C::kRowBytes;
      st = st + 1 == ST ? 0 : st + 1;
      const uint32_t valid = there[0];
#pragma unroll
      for (int i = 0; i + 1 < ST; ++i) there[i] = there[i + 1];
      // S^T: tokens rq, rq + 8 by vectors 8 n + 2 c + {0, 1}, in two chains each
      float sc[NQ][2][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) sc[n][k][0] = sc[n][k][1] = sc[n][k][2] = sc[n][k][3] = 0.f;
#pragma unroll
      for (int i = 0; i < C::kKP; ++i) {
        // (rows rq and rq + 8 have the same swizzle)
        const uint8_t* at = krows + rq * D + (((c + 4 * i) ^ k_swz(rq)) * 16);
        const uint4 k0 = *reinterpret_cast<const uint4*>(at);
        const uint4 k1 = *reinterpret_cast<const uint4*>(at + 8 * D);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a[4];
          fp8x4_to_f16<FMT>(word(k0, w), a[0], a[2]);
          fp8x4_to_f16<FMT>(word(k1, w), a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const uint2 q = C::kQRegs ? qb[n][C::kQRegs ? i * 4 + w : 0] : q_frag(n, i, w);
            mma16816(sc[n][w & 1], a, q.x, q.y);
          }
        }
      }
      // base-2 logits x[n][half][e]; tokens that a vector does not see by selection
      float x[NQ][2][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) x[n][h][e] = (sc[n][0][2 * h + e] + sc[n][1][2 * h + e]) * cq[n][e];
      if (valid != 0xFFFFu || t + kBlk > hi_min || !(t >= lo_max || t + kBlk <= span.sk)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = rq + 8 * h, v = t + k;
              const bool sees = ((valid >> k) & 1u) && v < row[n][e].hi && (v >= row[n][e].lo || v < span.sk);
              if (!sees) x[n][h][e] = -INFINITY;
            }
      }
      bool moves = false;
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y = fmaxf(x[n][0][e], x[n][1][e]);
          moves |= y - m[n][e] > kChunkTau;  // (false where both are -inf)
        }
      if (__any_sync(0xffffffffu, moves)) {
        // a vector's running maximum moves (whole numbers: rescaling is exact)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = fmaxf(x[n][0][e], x[n][1][e]);
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
            const float mo = m[n][e];
            const float mn = y - mo > kChunkTau ? fmaxf(mo, ceilf(y)) : mo;
            const float a = mn == mo ? 1.f : exp2_whole(mo - mn);
            m[n][e] = mn;
            l[n][e] *= a;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[i][n][e] *= a;
              o[i][n][2 + e] *= a;
            }
          }
      }
      // P^T: tokens 2 c + {0, 1} (+ 8) of vector 8 n + rq, as an fp16 number and the fp16 of
      // what that left: 2^-22 of p together, where one alone (2^-11) would be the largest error
      // of the call.  Up to 4 vectors: the second copy's columns carry the low halves.
      // More: products of their own.  (us with one half / so, 64 requests in a window of
      // 4096: 4 vectors 79.9 / 81.1, 8 vectors 80.6 / 85.4, 16 vectors 96.7 / 109; one request
      // of 8 vectors 7.3 / 7.5.)
      uint32_t pb[NQ][2], pl[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float s0 = __fadd_ru(m[n][0] == kNoMax ? 0.f : m[n][0], -kChunkPShift);
        const float s1 = __fadd_ru(m[n][1] == kNoMax ? 0.f : m[n][1], -kChunkPShift);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = fast_exp2(x[n][h][0] - s0), p1 = fast_exp2(x[n][h][1] - s1);
          l[n][0] += p0;
          l[n][1] += p1;
          const uint32_t hi = pack_half2(p0, p1);
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          const uint32_t lo = pack_half2(p0 - back.x, p1 - back.y);
          pb[n][h] = transpose8x8(TWIN && c >= 2 ? lo : hi);
          if (!TWIN) pl[n][h] = transpose8x8(lo);
        }
      }
#pragma unroll
      for (int i = 0; i < C::kVP; ++i) {
        uint4 vr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 2 * c + (j & 1) + 8 * (j >> 1);
          if (D >= 128) {
            vr[j] = *reinterpret_cast<const uint4*>(vrows + r * D + (((rq + 8 * i) ^ v_swz(r)) * 16));
          } else {
            const uint2 y =
                *reinterpret_cast<const uint2*>(vrows + r * D + (((rq >> 1) ^ v_swz(r)) * 16) + (rq & 1) * 8);
            vr[j] = make_uint4(y.x, y.y, 0u, 0u);
          }
        }
        if (valid != 0xFFFFu) {  // 0 * NaN of a token that is not there
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!((valid >> (2 * c + (j & 1) + 8 * (j >> 1))) & 1u)) vr[j] = make_uint4(0, 0, 0, 0);
        }
        if (zap) {
          constexpr bool e5 = FMT == FP8KV_KV_E5M2;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            vr[j] = make_uint4(zap_nonfinite(vr[j].x, e5), zap_nonfinite(vr[j].y, e5), zap_nonfinite(vr[j].z, e5),
                               zap_nonfinite(vr[j].w, e5));
        }
        // (the low halves' products go into the same sums a word later, behind other products)
        uint32_t f[2][2][4];  // [word parity][token pair][d of the word]
#pragma unroll
        for (int w = 0; w <= C::kVWords; ++w) {
          auto product = [&](int u, const uint32_t (&pp)[NQ][2]) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t (&g)[2][4] = f[u & 1];
              const uint32_t a[4] = {g[0][2 * k], g[0][2 * k + 1], g[1][2 * k], g[1][2 * k + 1]};
#pragma unroll
              for (int n = 0; n < NQ; ++n) mma16816(o[(i * C::kVWords + u) * 2 + k][n], a, pp[n][0], pp[n][1]);
            }
          };
          if (w < C::kVWords) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t wa = word(vr[2 * j], w), wb = word(vr[2 * j + 1], w);
              fp8x4_to_f16<FMT>(__byte_perm(wa, wb, 0x5140), f[w & 1][j][0], f[w & 1][j][1]);
              fp8x4_to_f16<FMT>(__byte_perm(wa, wb, 0x7362), f[w & 1][j][2], f[w & 1][j][3]);
            }
            product(w, pb);
          }
          if (!TWIN && w > 0) product(w - 1, pl);
        }
      }
    }
    cp_wait<0>();

    if (TWIN) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][0][k] += __shfl_xor_sync(0xffffffffu, o[i][0][k], 2);
    }

    // ---------------------------------------------------------- join the warps
    // (lane's vectors 8 n + 2 c + e; d tile (i, w, k) holds d = 128 i + PB rq + 4 w + 2 k + {0, 1})
    constexpr int PB = 4 * C::kVWords;           // bytes of a V piece
    float* sO = reinterpret_cast<float*>(ring);  // this warp's numerators [row][D]
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * c + e;
        float y = l[n][e];
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (rq == 0) {
          sML[warp * 32 + r] = m[n][e];
          sML[warp * 32 + 16 + r] = y;
        }
#pragma unroll
        for (int i = 0; i < C::kVP; ++i)
#pragma unroll
          for (int w = 0; w < C::kVWords; ++w) {
            const float (&lo)[4] = o[(i * C::kVWords + w) * 2][n], (&hi)[4] = o[(i * C::kVWords + w) * 2 + 1][n];
            *reinterpret_cast<float4*>(sO + r * D + 128 * i + PB * rq + 4 * w) =
                make_float4(lo[e], lo[2 + e], hi[e], hi[2 + e]);
          }
      }
    __syncthreads();
    float bad = 0.f;
#pragma unroll
    for (int k = 0; k < C::kIter; ++k) {
      const int x = tid + k * kThreadsS;
      const int r = x / (D / 4), d = (x % (D / 4)) * 4;
      acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      Ls[k] = 0.f;
      Ms[k] = kNoMax;
      if (r >= RC) continue;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) Ms[k] = fmaxf(Ms[k], sML[w * 32 + r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = sML[w * 32 + r], lw = sML[w * 32 + 16 + r];
        const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem + w * C::kRing) + r * D + d);
        // (a warp that saw nothing has a sum of 0 and numerators of 0)
        const float a = mw == Ms[k] ? 1.f : exp2_whole(mw - Ms[k]);
        Ls[k] = fmaf(a, lw, Ls[k]);
        acc[k].x = fmaf(a, y.x, acc[k].x);
        acc[k].y = fmaf(a, y.y, acc[k].y);
        acc[k].z = fmaf(a, y.z, acc[k].z);
        acc[k].w = fmaf(a, y.w, acc[k].w);
      }
      bad = fmaf(acc[k].x + acc[k].y + acc[k].z + acc[k].w, 0.f, bad);
    }
    if (zap) break;
    // Sums that are not finite: maybe only from codes of tokens that some rows do
    // not see (0 * NaN).  Once more without the non-finite V codes.
    if (!__syncthreads_or(bad != 0.f)) break;
    zap = true;
    fill([]() {});
  }

  if (zap) {
    uint32_t* kinds = reinterpret_cast<uint32_t*>(smem);  // non-finite marks [row][D]
    __syncthreads();
    mark_nonfinite_v<D, FMT>(p, kinds, b, g, u0, u1, span, RC,
                             [&](int i) { return chunk_row(p, req, span, token_of(i)); });
#pragma unroll
    for (int k = 0; k < C::kIter; ++k) {
      const int x = tid + k * kThreadsS;
      if (x / (D / 4) >= RC) continue;
      const uint32_t kd = kinds[x];
      float y[4] = {acc[k].x, acc[k].y, acc[k].z, acc[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((kd >> (8 * j)) & 0xFFu) y[j] = nonfinite_value((kd >> (8 * j)) & 0xFFu);
      acc[k] = make_float4(y[0], y[1], y[2], y[3]);
    }
  }
  auto out_at = [&](int r, int d) {
    return p.out + (int64_t)(req.row0 + token_of(r)) * p.o_st + (int64_t)head_of(r) * p.o_sh + d;
  };
  auto write_out = [&](uint16_t* to, const float4& y, float L) {
    const float f = vs / L;
    *reinterpret_cast<uint2*>(to) =
        L == 0.f ? make_uint2(0u, 0u) : make_uint2(pack_out<DT>(y.x * f, y.y * f), pack_out<DT>(y.z * f, y.w * f));
  };
  if (clustered) {
    // ---------------------------------------------------------- join the cluster
    const int run = div_s(p, C::kItems + p.S - 1);  // item x belongs to CTA x / run
    float2* pairs = reinterpret_cast<float2*>(smem + C::kOffPairs);
    float4* items = reinterpret_cast<float4*>(smem + C::kOffItems);
    __syncwarp();
    cluster_wait();
#pragma unroll
    for (int k = 0; k < C::kIter; ++k) {
      const int x = tid + k * kThreadsS, r = x / (D / 4);
      if (r >= RC) continue;
      int owner = 0;
#pragma unroll
      for (int q = 1; q < kChunkClusterMax; ++q) owner += x >= q * run;
      peer_store(peer_addr(items + s * run + (x - owner * run), owner), acc[k]);
      if (x % (D / 4) < p.S)  // one thread of the row per CTA
        peer_store(peer_addr(pairs + s * 16 + r, x % (D / 4)), make_float2(Ms[k], Ls[k]));
    }
    __syncwarp();
    cluster_arrive();
    // (the first item's place, while the others arrive)
    const int x0 = min(s * run + tid, C::kItems - 1);
    uint16_t* const to0 = out_at(x0 / (D / 4), (x0 % (D / 4)) * 4);
    cluster_wait();
    for (int i = tid; i < run; i += kThreadsS) {
      const int x = s * run + i, r = x / (D / 4), d = (x % (D / 4)) * 4;
      if (r >= RC) continue;
      // (all loads first; partitions past S read the last one's)
      float2 ml[kChunkClusterMax];
      float4 y[kChunkClusterMax];
#pragma unroll
      for (int q = 0; q < kChunkClusterMax; ++q) {
        const int at = min(q, p.S - 1);
        ml[q] = pairs[at * 16 + r];
        y[q] = items[at * run + i];
      }
      float M = kNoMax, L = 0.f;
#pragma unroll
      for (int q = 0; q < kChunkClusterMax; ++q) M = fmaxf(M, ml[q].x);
      float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kChunkClusterMax; ++q) {
        if (q >= p.S) continue;
        const float a = part_weight(ml[q].x, M);
        L = fmaf(a, ml[q].y, L);
        z.x = fmaf(a, y[q].x, z.x);
        z.y = fmaf(a, y[q].y, z.y);
        z.z = fmaf(a, y[q].z, z.z);
        z.w = fmaf(a, y[q].w, z.w);
      }
      write_out(i == tid ? to0 : out_at(r, d), z, L);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < C::kIter; ++k) {
    const int x = tid + k * kThreadsS;
    const int r = x / (D / 4), d = (x % (D / 4)) * 4;
    if (r >= RC) continue;
    if (p.S > 1) {
      if (d == 0) p.ml[s * plane + vec_of(r)] = make_float2(Ms[k], part_sum(Ls[k] * kChunkInvPShift));
      *reinterpret_cast<float4*>(p.partial + (s * plane + vec_of(r)) * D + d) =
          make_float4(acc[k].x * kChunkInvPShift, acc[k].y * kChunkInvPShift, acc[k].z * kChunkInvPShift,
                      acc[k].w * kChunkInvPShift);
    } else {
      write_out(out_at(r, d), acc[k], Ls[k]);
    }
  }
}

template <int D, int FMT, int DT, int NQ, bool TWIN>
cudaError_t run(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  auto fn = chunk_stream<D, FMT, DT, NQ, TWIN>;
  constexpr int smem = StreamCfg<D, NQ>::kSmem;
  static DeviceOnce once;
  cudaError_t e = once.run([&] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  const int chunks = (int)(((int64_t)p.max_q * p.G + kR - 1) / kR);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.Hkv), p.S, chunks);
  cfg.blockDim = dim3(kThreadsS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.y = p.S;
  attr.val.clusterDim.x = attr.val.clusterDim.z = 1;
  const bool clustered = chunk_clustered(plan);
  cfg.attrs = &attr;
  cfg.numAttrs = clustered ? 1 : 0;
  // (by_length takes up to 1 us: 13.9 us instead of 12.9 for 16 equal requests of 1000
  // positions, which this leaves out)
  const bool sorted = p.B <= kThreadsS && (int64_t)p.B * p.Hkv * p.S * chunks >= 2 * (int64_t)plan->num_sms &&
                      (p.window > 0 ? std::min(p.window, p.max_kv_len) : p.max_kv_len) >= 1024;
  return cudaLaunchKernelEx(&cfg, fn, p, (int)clustered, (int)sorted);
}

template <int D, int FMT, int DT>
cudaError_t pick_wide(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.max_q * p.G;
  if (rows > 8) return run<D, FMT, DT, 2, false>(plan, p, st);
  return rows > 4 ? run<D, FMT, DT, 1, false>(plan, p, st) : run<D, FMT, DT, 1, true>(plan, p, st);
}

template <int D>
cudaError_t pick(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  constexpr int E4 = FP8KV_KV_E4M3, E5 = FP8KV_KV_E5M2, F16 = FP8KV_DTYPE_F16, BF16 = FP8KV_DTYPE_BF16;
  if (plan->kv_format == E5)
    return plan->dtype == BF16 ? pick_wide<D, E5, BF16>(plan, p, st) : pick_wide<D, E5, F16>(plan, p, st);
  return plan->dtype == BF16 ? pick_wide<D, E4, BF16>(plan, p, st) : pick_wide<D, E4, F16>(plan, p, st);
}

}  // namespace

cudaError_t launch_chunk_stream(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  switch (plan->head_dim) {
    case 64: return pick<64>(plan, p, st);
    case 128: return pick<128>(plan, p, st);
    default: return pick<256>(plan, p, st);
  }
}

}  // namespace fp8kv
