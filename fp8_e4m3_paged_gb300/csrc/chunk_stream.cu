// Chunk attention for few query vectors (at most 16 per CTA: the query heads
// of one KV head times a few new tokens): bound by streaming the cache.
//
// One CTA of four warps per (request, KV head, 16 query vectors, partition);
// each warp walks blocks of 16 virtual tokens (chunk_span) on
// its own, and the four are joined at the end.  A block's FP8 bytes are
// requested a block or more ahead by cp.async into places of shared memory
// that only the requesting lane reads, so the loop has no barrier; each lane
// asks for the bytes that its MMA fragments hold:
//   S[16 x 8 tokens] = Q . K^T, m16n8k16: a lane of the B operand needs four
//     d of one token, so lane (n = lane/4, c = lane%4) loads the 16-byte pieces c, c + 4, ... of token n's row; each 32-bit word
//     decodes to one MMA's B fragment, and the d that a word holds is simply
//     the order in which Q's A fragments are laid out;
//   O[16 x D] += P . V: a B fragment needs two tokens of one d in a register,
//     so the lane loads the same 16-byte piece n of tokens 2c, 2c+1, 2c+8,
//     2c+9 (a warp reads whole rows) and interleaves their bytes before the
//     decode; P's fragment is what S's accumulators already hold.
// So a warp needs about 150 instructions per 4 KB of K and V.  Legacy
// mma.sync rather than tcgen05: with 4 to 16 useful rows the products are a
// few percent of the tensor peak, and TMEM or shared-memory operands would
// only add copies and barriers to a kernel whose time is the bytes' arrival.
//
// Partitions of one request and KV head form a thread-block cluster when there
// are at most 8: their sums are joined through distributed shared memory in
// the same launch.  More go through the workspace and chunk_join.
//
// With at most 8 query vectors the upper 8 rows of P's fragment are free:
// they carry P_lo = 2^11 (p - fp16(p)), which makes the probabilities good
// to 22 bits at no cost.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk_common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace fp8kv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreadsS = 32 * kWarps;
constexpr int kR = kChunkStreamRows;
constexpr float kLoUp = 2048.f, kLoDown = 1.f / 2048.f;

template <int D, bool WIDE>
struct StreamCfg {
  static constexpr int kRows = WIDE ? 16 : 8;
  static constexpr int kKP = D / 64;                 // 16-byte pieces of a K row per lane
  static constexpr int kVP = D >= 128 ? D / 128 : 1; // pieces of a V row per lane
  static constexpr int kVWords = D >= 128 ? 4 : 2;   // 32-bit words per piece
  static constexpr int kNT = D / 8;                  // n-tiles of O
  static constexpr int kQStride = D + 8;             // fp16 elements (padding: fragment loads without conflicts)
  static constexpr bool kQRegs = D <= 128;           // Q's fragments stay in registers
  static constexpr int kCtas = D == 256 ? 2 : D == 128 ? 3 : 5;  // resident per SM
  static constexpr int kBlk = kChunkStreamBlock; // positions per warp step
  static constexpr int kNB = kBlk / 16;              // ... in sub-blocks of an MMA's 16
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;  // blocks of a warp in flight or in use
  static constexpr int kKBytes = kNB * 2 * kKP * 512;  // a block's K pieces: [sub-block][piece][lane] of 16 bytes
  static constexpr int kVBytes = kNB * 4 * kVP * (D >= 128 ? 512 : 256);
  static constexpr int kRing = kStages * (kKBytes + kVBytes);  // per warp; then its numerators [row][D]
  static constexpr int kQBytes = kR * kQStride * 2;
  static constexpr int kOffQ = kWarps * kRing;
  static constexpr int kOffRed = kOffQ + kQBytes;    // per warp and row: maximum, sum; then inverse row scales
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

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async8(void* dst_smem, const void* src_gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(tc::smem_u32(dst_smem)), "l"(src_gmem) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Thread-block cluster: barrier over all its CTAs in two halves, and stores
// into a peer's shared memory (the place that `p` has in CTA `rank`).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
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

template <int D, int FMT, int DT, bool WIDE>
__global__ void __launch_bounds__(kThreadsS, StreamCfg<D, WIDE>::kCtas)
    chunk_stream(const __grid_constant__ ChunkParams p, const int clustered) {
  using C = StreamCfg<D, WIDE>;
  constexpr int ST = C::kStages, kBlk = C::kBlk, NB = C::kNB;
  constexpr uint32_t kAll = kBlk == 32 ? 0xFFFFFFFFu : 0xFFFFu;
  extern __shared__ __align__(16) uint8_t smem[];
  uint16_t* sQ = reinterpret_cast<uint16_t*>(smem + C::kOffQ);
  float* sM = reinterpret_cast<float*>(smem + C::kOffRed);  // [warp][16]
  float* sL = sM + kWarps * 16;
  float* sBack = sL + kWarps * 16;                          // [16] inverse row scales

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rq = lane >> 2, c = lane & 3;
  // KV heads next to each other, so that the CTAs that read one token's heads (adjacent
  // in memory) run at the same time
  const int g = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv, s = blockIdx.y;
  const int row_first = blockIdx.z * kR;  // packed rows: token * G + head of the group
  const ChunkRequest req = chunk_request(p, b);
  if (tid == 0 && req.bad) set_status(p.status, FP8KV_STATUS_BAD_LEN);
  const int RC = min(kR, req.n * p.G - row_first);
  if (RC <= 0) return;  // every CTA of the cluster
  if (clustered) cluster_arrive();  // peers may write here once all have come this far
  const int64_t plane = (int64_t)p.total_q * p.Hq;
  auto token_of = [&](int r) { return (row_first + r) / p.G; };
  auto head_of = [&](int r) { return g * p.G + (row_first + r) % p.G; };
  auto vec_of = [&](int r) { return (int64_t)(req.row0 + token_of(r)) * p.Hq + head_of(r); };

  const ChunkSpan span = chunk_span(p, req, token_of(0), token_of(RC - 1));
  int per = (span.U + p.S - 1) / p.S;
  per = (per + kBlk * kWarps - 1) / (kBlk * kWarps) * (kBlk * kWarps);
  const int u0 = (int)min((int64_t)s * per, (int64_t)span.U), u1 = min(span.U, u0 + per);
  if (u0 >= u1 && p.S > 1 && !clustered) {
    if (tid < RC) p.ml[s * plane + vec_of(tid)] = make_float2(kNoMax, 0.f);
    return;
  }

  // Places of a block's tokens, one per lane (of 16, both halves of the warp hold
  // them).  The block id is requested a block before it is needed; the copies
  // are unconditional (tokens without a place read the pool's first row and
  // are masked, V also zeroed).
  const uint8_t* kbase = p.k_cache + g * p.ksh + c * 16;
  const uint8_t* vbase = p.v_cache + g * p.vsh + rq * (D >= 128 ? 16 : 8);
  uint8_t* ring = smem + warp * C::kRing;
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
  // Copies of the block asked for into stage `st`; returns the tokens that are there.
  auto request = [&](const Ask& a, int st) {
    const bool ok = a.blk >= 0 && a.blk < p.num_kv_blocks;
    if (a.in && !ok) set_status(p.status, FP8KV_STATUS_BAD_BLOCK);
    const int64_t koff = ok ? a.blk * p.ksb + (int64_t)a.slot * p.kst : 0;
    const int64_t voff = ok ? a.blk * p.vsb + (int64_t)a.slot * p.vst : 0;
    uint8_t* dst = ring + st * (C::kKBytes + C::kVBytes);
#pragma unroll
    for (int h = 0; h < 2 * NB; ++h) {
      const uint8_t* src = kbase + __shfl_sync(0xffffffffu, koff, rq + 8 * h);
#pragma unroll
      for (int i = 0; i < C::kKP; ++i) tc::cp_async16(dst + ((h * C::kKP + i) * 32 + lane) * 16, src + 64 * i);
    }
    dst += C::kKBytes;
#pragma unroll
    for (int j = 0; j < 4 * NB; ++j) {
      const uint8_t* src = vbase + __shfl_sync(0xffffffffu, voff, 2 * c + (j & 1) + 8 * (j >> 1));
#pragma unroll
      for (int i = 0; i < C::kVP; ++i) {
        if (D >= 128)
          tc::cp_async16(dst + ((j * C::kVP + i) * 32 + lane) * 16, src + 128 * i);
        else
          cp_async8(dst + (j * 32 + lane) * 8, src);
      }
    }
    return __ballot_sync(0xffffffffu, ok) & kAll;
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
  constexpr int kQRows = kR / kWarps;
  uint32_t qw[kQRows][V / 2];
  const float ks = p.k_scale_dev ? __ldg(p.k_scale_dev) : p.k_scale;
  const float vs = p.v_scale_dev ? __ldg(p.v_scale_dev) : p.v_scale;
  fill([&]() {
#pragma unroll
    for (int k = 0; k < kQRows; ++k) {
      const int r = min(warp + k * kWarps, RC - 1);
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
      *reinterpret_cast<uint32_t*>(sQ + r * C::kQStride + lane * V + 2 * j) = r < RC ? w[j] ^ flip : 0u;
    if (lane == 0) sBack[r] = back;
  }
  __syncthreads();
  const float c0f = fabsf(cf) * sBack[rq], c1f = fabsf(cf) * sBack[rq + 8];

  // What this lane's two rows see; rows past RC see everything (their values are dropped).
  ChunkRow row0 = {INT_MAX, INT_MIN}, row1 = {INT_MAX, INT_MIN};
  if (rq < RC) row0 = chunk_row(p, req, span, token_of(rq));
  if (rq + 8 < RC) row1 = chunk_row(p, req, span, token_of(rq + 8));
  const int hi_min = __reduce_min_sync(0xffffffffu, min(row0.hi, row1.hi));
  const int lo_max = __reduce_max_sync(0xffffffffu, max(row0.lo, row1.lo));

  // Q's A fragments: step (i, w) covers d = 16 (c + 4 i) + 4 w + {0..3} of lane c
  auto q_frag = [&](int i, int w, uint32_t (&a)[4]) {
    const int d = (c + 4 * i) * 16 + 4 * w;
    const uint2 x = *reinterpret_cast<const uint2*>(sQ + rq * C::kQStride + d);
    a[0] = x.x;
    a[2] = x.y;
    if (WIDE) {
      const uint2 y = *reinterpret_cast<const uint2*>(sQ + (rq + 8) * C::kQStride + d);
      a[1] = y.x;
      a[3] = y.y;
    } else {
      a[1] = a[3] = 0u;
    }
  };
  uint32_t qa[C::kQRegs ? D / 16 : 1][4];
  if (C::kQRegs) {
#pragma unroll
    for (int i = 0; i < C::kKP; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) q_frag(i, w, qa[C::kQRegs ? i * 4 + w : 0]);
  }

  float o[C::kNT][4];
  float m0, m1, l0, l1;
  float4 acc[C::kIter];  // after the join: numerators of this thread's items, their rows' maxima and sums
  float Ms[C::kIter], Ls[C::kIter];
  bool zap = false;  // second pass: non-finite V codes enter as 0
  while (true) {
#pragma unroll
    for (int n = 0; n < C::kNT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    m0 = m1 = kNoMax;
    l0 = l1 = 0.f;
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
      const uint8_t* kst = ring + st * (C::kKBytes + C::kVBytes) + lane * 16;
      const uint8_t* vst = ring + st * (C::kKBytes + C::kVBytes) + C::kKBytes + lane * (D >= 128 ? 16 : 8);
      st = st + 1 == ST ? 0 : st + 1;
      const uint32_t valid = there[0];
#pragma unroll
      for (int i = 0; i + 1 < ST; ++i) there[i] = there[i + 1];
      float sc[2 * NB][4];  // [half sub-block]: 8 tokens
#pragma unroll
      for (int h = 0; h < 2 * NB; ++h) sc[h][0] = sc[h][1] = sc[h][2] = sc[h][3] = 0.f;
#pragma unroll
      for (int i = 0; i < C::kKP; ++i) {
        uint4 kr[2 * NB];
#pragma unroll
        for (int h = 0; h < 2 * NB; ++h) kr[h] = *reinterpret_cast<const uint4*>(kst + (h * C::kKP + i) * 512);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a[4];
          if (!C::kQRegs) q_frag(i, w, a);
#pragma unroll
          for (int h = 0; h < 2 * NB; ++h) {
            uint32_t b0, b1;
            fp8x4_to_f16<FMT>(word(kr[h], w), b0, b1);
            mma16816(sc[h], C::kQRegs ? qa[C::kQRegs ? i * 4 + w : 0] : a, b0, b1);
          }
        }
      }
      // base-2 logits; tokens that a row does not see by selection
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2 * NB; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[h][e] *= c0f;
          if (WIDE) sc[h][2 + e] *= c1f;
        }
      if (valid != kAll || t + kBlk > hi_min || !(t >= lo_max || t + kBlk <= span.sk)) {
#pragma unroll
        for (int h = 0; h < 2 * NB; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = 8 * h + 2 * c + e, v = t + x;
            const bool ok = (valid >> x) & 1u;
            if (!(ok && v < row0.hi && (v >= row0.lo || v < span.sk))) sc[h][e] = -INFINITY;
            if (WIDE && !(ok && v < row1.hi && (v >= row1.lo || v < span.sk))) sc[h][2 + e] = -INFINITY;
          }
      }
#pragma unroll
      for (int h = 0; h < 2 * NB; ++h) {
        x0 = fmaxf(fmaxf(x0, sc[h][0]), sc[h][1]);
        if (WIDE) x1 = fmaxf(fmaxf(x1, sc[h][2]), sc[h][3]);
      }
      if (__any_sync(0xffffffffu, (x0 > -INFINITY && !(x0 <= m0 + kChunkTau)) ||
                                      (x1 > -INFINITY && !(x1 <= m1 + kChunkTau)))) {
        // a row's running maximum moves (integers: rescaling is exact)
        float y0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, 2));
        float y1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, 2));
        const float n0 = y0 > m0 + kChunkTau || m0 == kNoMax ? fmaxf(m0, ceilf(y0)) : m0;
        const float n1 = y1 > m1 + kChunkTau || m1 == kNoMax ? fmaxf(m1, ceilf(y1)) : m1;
        const float a0 = n0 == m0 ? 1.f : exp2_whole(m0 - n0), a1 = n1 == m1 ? 1.f : exp2_whole(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
          o[n][0] *= a0;
          o[n][1] *= a0;
          o[n][2] *= WIDE ? a1 : a0;
          o[n][3] *= WIDE ? a1 : a0;
        }
      }
      const float s0 = (m0 == kNoMax ? 0.f : m0) - kChunkPShift, s1 = (m1 == kNoMax ? 0.f : m1) - kChunkPShift;
      uint32_t pa[NB][4];
#pragma unroll
      for (int h = 0; h < 2 * NB; ++h) {
        uint32_t* q = &pa[h / 2][2 * (h & 1)];
        const float p0 = fast_exp2(sc[h][0] - s0), p1 = fast_exp2(sc[h][1] - s0);
        l0 += p0 + p1;
        q[0] = pack_half2(p0, p1);
        if (WIDE) {
          const float p2 = fast_exp2(sc[h][2] - s1), p3 = fast_exp2(sc[h][3] - s1);
          l1 += p2 + p3;
          q[1] = pack_half2(p2, p3);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<__half2*>(&q[0]));
          q[1] = pack_half2((p0 - f.x) * kLoUp, (p1 - f.y) * kLoUp);
        }
      }
#pragma unroll
      for (int sb = 0; sb < NB; ++sb)
#pragma unroll
        for (int i = 0; i < C::kVP; ++i) {
          uint4 vr[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (D >= 128) {
              vr[j] = *reinterpret_cast<const uint4*>(vst + ((4 * sb + j) * C::kVP + i) * 512);
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(vst + (4 * sb + j) * 256);
              vr[j] = make_uint4(y.x, y.y, 0u, 0u);
            }
          }
          if (valid != kAll) {  // 0 * NaN of a token that is not there
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!((valid >> (16 * sb + 2 * c + (j & 1) + 8 * (j >> 1))) & 1u)) vr[j] = make_uint4(0, 0, 0, 0);
          }
          if (zap) {
            constexpr bool e5 = FMT == FP8KV_KV_E5M2;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              vr[j] = make_uint4(zap_nonfinite(vr[j].x, e5), zap_nonfinite(vr[j].y, e5), zap_nonfinite(vr[j].z, e5),
                                 zap_nonfinite(vr[j].w, e5));
          }
#pragma unroll
          for (int w = 0; w < C::kVWords; ++w) {
            uint32_t f[2][4];  // [token pair][d of the word]
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t wa = word(vr[2 * j], w), wb = word(vr[2 * j + 1], w);
              fp8x4_to_f16<FMT>(__byte_perm(wa, wb, 0x5140), f[j][0], f[j][1]);
              fp8x4_to_f16<FMT>(__byte_perm(wa, wb, 0x7362), f[j][2], f[j][3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) mma16816(o[(i * C::kVWords + w) * 4 + e], pa[sb], f[0][e], f[1][e]);
          }
        }
    }
    cp_wait<0>();

    // ---------------------------------------------------------- join the warps
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (c == 0) {
      sM[warp * 16 + rq] = m0;
      sL[warp * 16 + rq] = l0;
      if (WIDE) {
        sM[warp * 16 + rq + 8] = m1;
        sL[warp * 16 + rq + 8] = l1;
      }
    }
    // n-tile (i, x) column n of O is d = 128 i + PB n + x, PB the bytes of a V piece
    constexpr int PB = 4 * C::kVWords;
    float* sO = reinterpret_cast<float*>(ring);  // this warp's numerators [row][D]
#pragma unroll
    for (int i = 0; i < C::kVP; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 0; x < PB; x += 4) {
          const int d = 128 * i + PB * (2 * c + e) + x;
          float f[4], h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[k] = o[i * PB + x + k][e];
            h[k] = o[i * PB + x + k][2 + e];
            if (!WIDE) f[k] = fmaf(h[k], kLoDown, f[k]);
          }
          *reinterpret_cast<float4*>(sO + rq * D + d) = make_float4(f[0], f[1], f[2], f[3]);
          if (WIDE) *reinterpret_cast<float4*>(sO + (rq + 8) * D + d) = make_float4(h[0], h[1], h[2], h[3]);
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
      for (int w = 0; w < kWarps; ++w) Ms[k] = fmaxf(Ms[k], sM[w * 16 + r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = sM[w * 16 + r], lw = sL[w * 16 + r];
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
  auto write_out = [&](int r, int d, const float4& y, float L) {
    const float f = vs / L;
    *reinterpret_cast<uint2*>(p.out + (int64_t)(req.row0 + token_of(r)) * p.o_st + (int64_t)head_of(r) * p.o_sh + d) =
        L == 0.f ? make_uint2(0u, 0u) : make_uint2(pack_out<DT>(y.x * f, y.y * f), pack_out<DT>(y.z * f, y.w * f));
  };
  if (clustered) {
    // ---------------------------------------------------------- join the cluster
    const int run = (C::kItems + p.S - 1) / p.S;  // item x belongs to CTA x / run
    float2* pairs = reinterpret_cast<float2*>(smem + C::kOffPairs);
    float4* items = reinterpret_cast<float4*>(smem + C::kOffItems);
    __syncwarp();
    cluster_wait();
#pragma unroll
    for (int k = 0; k < C::kIter; ++k) {
      const int x = tid + k * kThreadsS, r = x / (D / 4);
      if (r >= RC) continue;
      const int owner = x / run;
      peer_store(peer_addr(items + s * run + (x - owner * run), owner), acc[k]);
      if (x % (D / 4) == 0)
        for (int q = 0; q < p.S; ++q) peer_store(peer_addr(pairs + s * 16 + r, q), make_float2(Ms[k], Ls[k]));
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (int i = tid; i < run; i += kThreadsS) {
      const int x = s * run + i, r = x / (D / 4), d = (x % (D / 4)) * 4;
      if (r >= RC) continue;
      float M = kNoMax, L = 0.f;
      for (int q = 0; q < p.S; ++q) M = fmaxf(M, pairs[q * 16 + r].x);
      float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < p.S; ++q) {
        const float2 ml = pairs[q * 16 + r];
        const float4 y = items[q * run + i];
        if (ml.x == kNoMax && ml.y == 0.f) continue;  // saw nothing
        const float a = part_weight(ml.x, M);
        L = fmaf(a, ml.y, L);
        z.x = fmaf(a, y.x, z.x);
        z.y = fmaf(a, y.y, z.y);
        z.z = fmaf(a, y.z, z.z);
        z.w = fmaf(a, y.w, z.w);
      }
      write_out(r, d, z, L);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < C::kIter; ++k) {
    const int x = tid + k * kThreadsS;
    const int r = x / (D / 4), d = (x % (D / 4)) * 4;
    if (r >= RC) continue;
    if (p.S > 1) {
      if (d == 0) p.ml[s * plane + vec_of(r)] = make_float2(Ms[k], Ls[k] * kChunkInvPShift);
      *reinterpret_cast<float4*>(p.partial + (s * plane + vec_of(r)) * D + d) =
          make_float4(acc[k].x * kChunkInvPShift, acc[k].y * kChunkInvPShift, acc[k].z * kChunkInvPShift,
                      acc[k].w * kChunkInvPShift);
    } else {
      write_out(r, d, acc[k], Ls[k]);
    }
  }
}

template <int D, int FMT, int DT, bool WIDE>
cudaError_t run(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  auto fn = chunk_stream<D, FMT, DT, WIDE>;
  constexpr int smem = StreamCfg<D, WIDE>::kSmem;
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
  return cudaLaunchKernelEx(&cfg, fn, p, (int)clustered);
}

template <int D, int FMT, int DT>
cudaError_t pick_wide(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  return (int64_t)p.max_q * p.G > 8 ? run<D, FMT, DT, true>(plan, p, st) : run<D, FMT, DT, false>(plan, p, st);
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
