// Gathered weights for few query vectors (decode steps, short drafts: 16 per CTA and KV head), and for more
// of them on few positions.
//
//   x_rt = c q_r . k_t (base 2),  p_rt = 2^(x_rt - M_r) / L_r,  score_t = decay score_t + sum_r p_rt
//
// M_r and L_r are known only when every position has been seen.  The first kernel therefore
// streams K once (the bytes that bound the call), keeps the logits, which for 4 vectors are 16 bytes
// beside a row of 128, and leaves each partition's maxima and sums; the second adds the
// logits' weights up per position.  Reading K a second time instead would double the bytes.
//
// First kernel: one CTA of four warps per (request, KV head, partition); each warp walks
// blocks of 32 positions on its own, rows requested by cp.async into its ring, a lane for each row's
// place.  (Blocks of 16, one chain of products and exponentials at a time, took 2400 cycles each with
// four warps on a scheduler: 60 us for 64 requests of 4000 positions.)
// 64 requests of 512 to 16000 positions, 32 heads over 8, D 128: 80 us with the second kernel (59 % of the bytes'
// time at the copy rate), of which this one takes 65: four warps' chains on each scheduler, not DRAM, bound it.
// One request of 4001: 7.1 us, two launches and the chain lengths -> block table -> rows.
// S^T[16 tokens x 8 vectors] = K . Q^T by mma.sync m16n8k16: lane (n = lane/4, c = lane%4) of
// the A operand takes the 16-byte pieces c, c + 4, ... of rows n and n + 8, a word of each decodes to
// one fragment, and Q's B fragments are laid out in that order of d.
#include <algorithm>
#include <climits>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "score_common.cuh"
#include "stream_ptx.cuh"
#include "tc_ptx.cuh"

namespace fp8kv {
namespace {

constexpr int kWarps = kChunkStreamWarps;
constexpr int kThreadsS = 32 * kWarps;
constexpr int kBlk = 32;                            // positions of a warp's block
constexpr int kSub = kBlk / 16;                     // ... in MMAs of 16
constexpr int kFoldThreads = 256;
// positions of a thread of the second kernel
constexpr int fold_each(int vectors) { return vectors == 16 ? 2 : 4; }

template <int D, int NQ>
struct Cfg {
  static constexpr int kKP = D / 64;                 // 16-byte pieces of a row per lane
  static constexpr int kQStride = D + 8;             // fp16 elements (padding: fragment loads without conflicts)
  static constexpr bool kQRegs = D * NQ <= 256;      // Q's fragments stay in registers
  static constexpr int kCtas = D == 256 ? 3 : 4;     // resident per SM
  static constexpr int kStages = D == 64 ? 5 : D == 128 ? 3 : 2;
  static constexpr int kCh = D / 16;                 // 16-byte pieces of a row, lanes that copy it
  static constexpr int kRowsIt = 32 / kCh;           // rows that the warp copies at a time
  static constexpr int kRowBytes = kBlk * D;         // a block's rows
  static constexpr int kRing = kStages * kRowBytes;  // per warp
  static constexpr int kOffQ = kWarps * kRing;
  static constexpr int kOffRed = kOffQ + 8 * NQ * kQStride * 2;  // per warp: row offsets, then maxima and sums
  static constexpr int kSmem = kOffRed + kWarps * kBlk * 8 + 16 * 4;
};

template <int D, int FMT, int DT, int NQ>
__global__ void __launch_bounds__(kThreadsS, Cfg<D, NQ>::kCtas)
    score_logits(const __grid_constant__ ScoreParams sp) {
  using C = Cfg<D, NQ>;
  constexpr int ST = C::kStages, R = 8 * NQ;
  const ChunkParams& p = sp.c;
  extern __shared__ __align__(16) uint8_t smem[];
  uint16_t* sQ = reinterpret_cast<uint16_t*>(smem + C::kOffQ);
  float* sML = reinterpret_cast<float*>(smem + C::kOffRed);  // [warp][64]: 16 maxima, then 16 sums
  float* sBack = sML + kWarps * kBlk * 2;                    // [16] inverse row scales

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rq = lane >> 2, c = lane & 3;
  let_next_kernel_start();
  const int b = div_hkv(p, blockIdx.x), g = blockIdx.x - b * p.Hkv, s = blockIdx.y;
  const ChunkRequest req = chunk_request(p, b);
  if (tid == 0 && req.bad) set_status(p.status, FP8KV_STATUS_BAD_LEN);
  const int row_first = blockIdx.z * kScoreGroupRows;
  const int RC = min(R, req.n * p.G - row_first);
  if (RC <= 0) return;
  const int64_t plane = (int64_t)p.total_q * p.Hq;
  auto token_of = [&](int r) { return token_at(p, row_first + r); };
  auto head_of = [&](int r) { return g * p.G + row_at(p, row_first + r).head; };
  auto vec_of = [&](int r) { return (int64_t)(req.row0 + token_of(r)) * p.Hq + head_of(r); };
  // (partitions of one length, whatever the request's: a batch of 64 between 512 and 16000 positions,
  // whose longest CTAs had 16000, took 160 us)
  const int u0 = (int)min((int64_t)s * sp.stat_part, (int64_t)req.kv);
  const int u1 = (int)min((int64_t)u0 + sp.stat_part, (int64_t)req.kv);
  if (u0 >= u1) return;  // (nor does the second kernel read it)

  // (as in the attention's streaming kernel, block ids one block ahead; rows of tokens without a
  // place are zeros, and masked)
  const uint8_t* kbase = p.k_cache + g * p.ksh + (lane % C::kCh) * 16;
  uint8_t* ring = smem + warp * C::kRing;
  int64_t* place = reinterpret_cast<int64_t*>(sML + warp * 64);
  static_assert(kBlk * 8 == 64 * 4, "one in place of the other");
  struct Ask {
    int blk, slot;
    bool in;
  };
  auto ask = [&](int t) {
    const int v = t + lane;
    Ask a = {-1, 0, v < u1};
    if (a.in) {
      const int page = div_page(v, p.page_size, p.page_div);
      a.slot = v - page * p.page_size;
      a.blk = __ldg(p.block_table + (int64_t)b * p.bt_stride + page);
    }
    return a;
  };
  auto swz = [](int r) { return D >= 128 ? 4 * (r & 1) : 0; };
  auto request = [&](const Ask& a, int st) {
    const bool ok = a.blk >= 0 && a.blk < p.num_kv_blocks;
    if (a.in && !ok) set_status(p.status, FP8KV_STATUS_BAD_BLOCK);
    const uint32_t rows = __ballot_sync(0xffffffffu, ok);
    place[lane] = ok ? a.blk * p.ksb + (int64_t)a.slot * p.kst : 0;
    __syncwarp();
    uint8_t* dst = ring + st * C::kRowBytes;
#pragma unroll
    for (int it = 0; it < kBlk / C::kRowsIt; ++it) {
      const int r = it * C::kRowsIt + lane / C::kCh;
      tc::cp_async16_or_zero(dst + r * D + (((lane % C::kCh) ^ swz(r)) * 16), kbase + place[r], (rows >> r) & 1u ? 16u : 0u);
    }
    __syncwarp();
    return rows;
  };
  constexpr int kStep = kBlk * kWarps;
  const int t_first = u0 + kBlk * warp;
  uint32_t there[ST];  // tokens of the blocks in flight, the oldest first
  Ask first[ST];
#pragma unroll
  for (int i = 0; i < ST; ++i) first[i] = ask(t_first + i * kStep);
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) {
    there[i] = t_first + i * kStep < u1 ? request(first[i], i) : 0u;
    cp_commit();
  }
  Ask next = first[ST - 1];

  // Q -> shared memory as fp16 (bf16 rows scaled by a power of two); rows past RC are zero
  constexpr int V = D / 32;  // elements per lane
  const float ks = p.k_scale_dev ? __ldg(p.k_scale_dev) : p.k_scale;
  const float cf = p.softmax_scale * ks * kLog2e;
  const uint32_t flip = cf < 0.f ? 0x80008000u : 0u;  // logit factors are non-negative from here on
#pragma unroll
  for (int r = warp; r < R; r += kWarps) {
    const int rr = min(r, RC - 1);
    const uint16_t* src = p.q + (int64_t)(req.row0 + token_of(rr)) * p.q_st + (int64_t)head_of(rr) * p.q_sh;
    uint32_t w[V / 2];
    if constexpr (V == 2)
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(src) + lane);
    else if constexpr (V == 4)
      *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(src) + lane);
    else
      *reinterpret_cast<uint4*>(w) = __ldg(reinterpret_cast<const uint4*>(src) + lane);
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

  // This lane's vectors 8 n + 2 c + e: logit factors, and how far they see (vectors past RC: not at all)
  float cq[NQ][2];
  int hi[NQ][2], hi_min = INT_MAX;
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * c + e;
      cq[n][e] = fabsf(cf) * sBack[r];
      hi[n][e] = r < RC ? req.kv - req.n + token_of(r) + 1 : INT_MIN;
      // (a column that no vector has stays out of the test for whole blocks: its logits are 0, and
      // what is kept of them is not read)
      if (r < RC) hi_min = min(hi_min, hi[n][e]);
    }
  hi_min = __reduce_min_sync(0xffffffffu, hi_min);

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

  float m[NQ][2], l[NQ][2];  // running maxima (whole numbers, base 2); sums over this lane's tokens
#pragma unroll
  for (int n = 0; n < NQ; ++n) m[n][0] = m[n][1] = kNoMax, l[n][0] = l[n][1] = 0.f;
  const int RV = sp.vectors;
  float* keep = sp.logits + ((int64_t)b * p.Hkv + g) * p.max_kv_len * RV + row_first + 2 * c;
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
    const uint8_t* krows = ring + st * C::kRowBytes;
    st = st + 1 == ST ? 0 : st + 1;
    const uint32_t valid = there[0];
#pragma unroll
    for (int i = 0; i + 1 < ST; ++i) there[i] = there[i + 1];
    float sc[NQ][kSub][2][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int k = 0; k < 2; ++k) sc[n][u][k][0] = sc[n][u][k][1] = sc[n][u][k][2] = sc[n][u][k][3] = 0.f;
#pragma unroll
    for (int i = 0; i < C::kKP; ++i) {
      uint4 k0[kSub], k1[kSub];
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const uint8_t* at = krows + (16 * u + rq) * D + (((c + 4 * i) ^ swz(rq)) * 16);
        k0[u] = *reinterpret_cast<const uint4*>(at);
        k1[u] = *reinterpret_cast<const uint4*>(at + 8 * D);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          uint32_t a[4];
          fp8x4_to_f16<FMT>(word(k0[u], w), a[0], a[2]);
          fp8x4_to_f16<FMT>(word(k1[u], w), a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const uint2 q = C::kQRegs ? qb[n][C::kQRegs ? i * 4 + w : 0] : q_frag(n, i, w);
            mma16816(sc[n][u][w & 1], a, q.x, q.y);
          }
        }
    }
    float x[NQ][2 * kSub][2];  // [.][16-row half][.]
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int h = 0; h < 2 * kSub; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e)  // (rounded: the maximum is of these numbers, and they are what is kept)
          x[n][h][e] = __fmul_rn(sc[n][h / 2][0][2 * (h & 1) + e] + sc[n][h / 2][1][2 * (h & 1) + e], cq[n][e]);
    if (valid != 0xFFFFFFFFu || t + kBlk > hi_min) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int h = 0; h < 2 * kSub; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = rq + 8 * h;
            if (!((valid >> k) & 1u) || t + k >= hi[n][e]) x[n][h][e] = -INFINITY;
          }
    }
    auto top = [&](int n, int e) {
      float y = x[n][0][e];
#pragma unroll
      for (int h = 1; h < 2 * kSub; ++h) y = fmaxf(y, x[n][h][e]);
      return y;
    };
    bool moves = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) moves |= top(n, e) - m[n][e] > kChunkTau;
    if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = top(n, e);
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
          const float mo = m[n][e];
          const float mn = y - mo > kChunkTau ? fmaxf(mo, ceilf(y)) : mo;
          m[n][e] = mn;
          l[n][e] *= mn == mo ? 1.f : exp2_whole(mo - mn);
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float s0 = m[n][0] == kNoMax ? 0.f : m[n][0], s1 = m[n][1] == kNoMax ? 0.f : m[n][1];
#pragma unroll
      for (int h = 0; h < 2 * kSub; ++h) {
        l[n][0] += fast_exp2(x[n][h][0] - s0);
        l[n][1] += fast_exp2(x[n][h][1] - s1);
        const int tt = t + rq + 8 * h;
        if (row_first + 8 * n + 2 * c < RV && tt < u1)
          *reinterpret_cast<float2*>(keep + (int64_t)tt * RV + 8 * n) = make_float2(x[n][h][0], x[n][h][1]);
      }
    }
  }
  cp_wait<0>();
  // join the warps (the offsets' places become maxima and sums: each warp its own)
  __syncwarp();
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
        sML[warp * 64 + r] = m[n][e];
        sML[warp * 64 + 16 + r] = y;
      }
    }
  __syncthreads();
  if (tid < RC) {
    float M = kNoMax, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sML[w * 64 + tid]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = sML[w * 64 + tid], lw = sML[w * 64 + 16 + tid];
      if (lw != 0.f) L = fmaf(part_weight(mw, M), lw, L);
    }
    p.ml[s * plane + vec_of(tid)] = make_float2(M, L);
  }
}

// Position t, its weight written, becomes NaN if a vector with a NaN sum sees it, also where that vector's own logit is
// -inf: which is what is kept, too, where a vector does not see the position, so lengths and table tell them apart.  (Behind
// the sums, since in their midst it took 3 to 10 us of a batch's 80.)
__device__ __forceinline__ void pass_nan_on(const ScoreParams& sp, const Norm* norm, int RC, int b, int g, int base, int t) {
  int64_t blk;
  int slot;
  if (!chunk_place(sp.c, b, t, blk, slot)) return;
#pragma unroll 1
  for (int r = 0; r < RC; ++r)
    if (norm[r].inv != norm[r].inv && t <= base + token_at(sp.c, r)) sp.out[b * sp.out_sr + g * sp.out_sh + t] = norm[r].inv;
}
// Whether there is such a vector.
__device__ __forceinline__ bool any_nan(const Norm* norm, int n) {
  bool nan = false;
  for (int r = 0; r < n; ++r) nan |= norm[r].inv != norm[r].inv;
  return nan;
}

// Second kernel: a few positions per thread.
// (CTAs of an SM as without the look for NaN, which took more registers: 82 us for a batch's 80)
template <int RV>
__global__ void __launch_bounds__(kFoldThreads, RV == 4 ? 8 : RV == 8 ? 4 : 5) score_fold(const __grid_constant__ ScoreParams sp) {
  constexpr int EACH = fold_each(RV);
  const ChunkParams& p = sp.c;
  __shared__ Norm norm[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = div_hkv(p, blockIdx.y), g = blockIdx.y - b * p.Hkv;
  const ChunkRequest req = chunk_request(p, b);
  const int RC = min(RV, req.n * p.G), base = req.kv - req.n;
  const int t0 = (int)min((int64_t)blockIdx.x * kFoldThreads * EACH, (int64_t)req.kv);
  if (RC <= 0 || t0 >= req.kv) {
    leave_in_order();
    return;
  }
  wait_for_previous_kernel();
  const int S = (req.kv - 1) / sp.stat_part + 1;
  for (int r = warp; r < RV; r += kFoldThreads / 32) {
    Norm n = {0.f, 0.f};
    if (r < RC) {
      const RowAt at = row_at(p, r);
      n = join_norm(p.ml, (int64_t)p.total_q * p.Hq, (int64_t)(req.row0 + at.token) * p.Hq + g * p.G + at.head, S, lane, 32);
    }
    if (lane == 0) norm[r] = n;
  }
  const float4* from = reinterpret_cast<const float4*>(sp.logits + ((int64_t)b * p.Hkv + g) * p.max_kv_len * RV);
  float4 y[EACH][RV / 4];
#pragma unroll
  for (int j = 0; j < EACH; ++j)
#pragma unroll
    for (int i = 0; i < RV / 4; ++i)  // (past the last position: read again, not used)
      y[j][i] = __ldcg(from + (int64_t)min(t0 + j * kFoldThreads + tid, req.kv - 1) * (RV / 4) + i);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int t = t0 + j * kFoldThreads + tid;
    if (t >= req.kv) break;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < RV / 4; ++i) {
      const float z[4] = {y[j][i].x, y[j][i].y, y[j][i].z, y[j][i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 4 * i + k;
        // (a position that the vector does not see, or a column without a vector, adds nothing, NaN sums included)
        if (r < RC && z[k] != -INFINITY) sum = fmaf(fast_exp2(z[k] - norm[r].m), norm[r].inv, sum);
      }
    }
    write_score(sp, b, g, t, base, sum);
  }
  if (any_nan(norm, RV)) {
#pragma unroll 1
    for (int j = 0; j < EACH; ++j) {
      const int t = t0 + j * kFoldThreads + tid;
      if (t < req.kv) pass_nan_on(sp, norm, RC, b, g, base, t);
    }
  }
}

// More than 16 vectors: `lanes` neighbouring threads per position (a power of two), 16 vectors each.
__global__ void __launch_bounds__(kFoldThreads) score_fold_many(const __grid_constant__ ScoreParams sp, const int lanes) {
  const ChunkParams& p = sp.c;
  __shared__ Norm norm[kScoreStreamRows];
  static_assert(kScoreStreamRows == kFoldThreads, "a thread for each vector's sum");
  const int tid = threadIdx.x, RV = sp.vectors;
  const int b = div_hkv(p, blockIdx.y), g = blockIdx.y - b * p.Hkv;
  const ChunkRequest req = chunk_request(p, b);
  const int RC = min(RV, req.n * p.G), base = req.kv - req.n;
  const int each = kFoldThreads / lanes, t0 = (int)min((int64_t)blockIdx.x * each, (int64_t)req.kv);
  if (RC <= 0 || t0 >= req.kv) {
    leave_in_order();
    return;
  }
  wait_for_previous_kernel();
  const int t = t0 + tid / lanes, r0 = (tid & (lanes - 1)) * kScoreGroupRows;
  // (positions past the last one and vectors past RV: read again, not used)
  const float4* from = reinterpret_cast<const float4*>(
      sp.logits + (((int64_t)b * p.Hkv + g) * p.max_kv_len + min(t, req.kv - 1)) * RV + min(r0, RV - kScoreGroupRows));
  float4 y[kScoreGroupRows / 4];
#pragma unroll
  for (int i = 0; i < kScoreGroupRows / 4; ++i) y[i] = __ldcg(from + i);
  Norm mine = {0.f, 0.f};
  if (tid < RC) {
    const RowAt at = row_at(p, tid);
    mine = join_norm(p.ml, (int64_t)p.total_q * p.Hq, (int64_t)(req.row0 + at.token) * p.Hq + g * p.G + at.head,
                     (req.kv - 1) / sp.stat_part + 1);
  }
  norm[tid] = mine;
  const bool nan = __syncthreads_or(mine.inv != mine.inv);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kScoreGroupRows / 4; ++i) {
    const float z[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + 4 * i + k;
      if (r < RC && z[k] != -INFINITY) sum = fmaf(fast_exp2(z[k] - norm[r].m), norm[r].inv, sum);
    }
  }
  for (int o = lanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (t >= req.kv || r0 != 0) return;
  write_score(sp, b, g, t, base, sum);
  if (nan) pass_nan_on(sp, norm, RC, b, g, base, t);
}

template <int D, int FMT, int DT, int NQ>
cudaError_t run(const ScoreParams& p, cudaStream_t st) {
  auto fn = score_logits<D, FMT, DT, NQ>;
  constexpr int smem = Cfg<D, NQ>::kSmem;
  static DeviceOnce once;
  cudaError_t e = once.run([&] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  const unsigned pairs = (unsigned)(p.c.B * p.c.Hkv);
  fn<<<dim3(pairs, p.c.S, (p.vectors + kScoreGroupRows - 1) / kScoreGroupRows), kThreadsS, smem, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.vectors > kScoreGroupRows) {
    int lanes = 2;
    while (lanes * kScoreGroupRows < p.vectors) lanes *= 2;
    const int each = kFoldThreads / lanes;
    return launch_dependent(score_fold_many, dim3((unsigned)((p.c.max_kv_len + each - 1) / each), pairs), kFoldThreads, 0,
                            st, p, lanes);
  }
  const int each = kFoldThreads * fold_each(p.vectors);
  const dim3 grid((unsigned)((p.c.max_kv_len + each - 1) / each), pairs);
  return launch_dependent(p.vectors == 4 ? score_fold<4> : p.vectors == 8 ? score_fold<8> : score_fold<16>, grid,
                          kFoldThreads, 0, st, p);
}

template <int D, int FMT, int DT>
cudaError_t pick_width(const ScoreParams& p, cudaStream_t st) {
  return p.vectors > 8 ? run<D, FMT, DT, 2>(p, st) : run<D, FMT, DT, 1>(p, st);
}

template <int D>
cudaError_t pick(const fp8kv_cache_score_plan_t* plan, const ScoreParams& p, cudaStream_t st) {
  constexpr int E4 = FP8KV_KV_E4M3, E5 = FP8KV_KV_E5M2, F16 = FP8KV_DTYPE_F16, BF16 = FP8KV_DTYPE_BF16;
  if (plan->kv_format == E5)
    return plan->dtype == BF16 ? pick_width<D, E5, BF16>(p, st) : pick_width<D, E5, F16>(p, st);
  return plan->dtype == BF16 ? pick_width<D, E4, BF16>(p, st) : pick_width<D, E4, F16>(p, st);
}

}  // namespace

cudaError_t launch_score_stream(const fp8kv_cache_score_plan_t* plan, const ScoreParams& p, cudaStream_t st) {
  switch (plan->head_dim) {
    case 64: return pick<64>(plan, p, st);
    case 128: return pick<128>(plan, p, st);
    default: return pick<256>(plan, p, st);
  }
}

}  // namespace fp8kv
