// Geometry and small device helpers shared by the chunk-attention kernels.
#pragma once

#include <climits>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "chunk.h"
#include "device_common.cuh"

namespace fp8kv {

constexpr float kChunkTau = 8.0f;              // the running maximum moves when a logit exceeds it by 2^tau
constexpr float kChunkPShift = 7.0f;           // probabilities are kept times 2^7: p <= 2^15 fits fp16, and
constexpr float kChunkInvPShift = 1.f / 128;   // p turns subnormal only below 2^-21 of the running maximum
constexpr float kNoMax = -INFINITY;            // running maximum of a row that has seen nothing
// Logits of 2^24 and more are so far apart that m + tau and m - 7 round: p must not pass
// 2^15 for it (fp16 ends at 2^16).  Differences of near numbers are exact, so the maximum
// moves by logit - m > tau, and the shift is rounded to the side of the smaller p.

// Packed row -> token of the request and query head of the group; partitions' length;
// KV head of a CTA.  By products with host-made inverses, for the stream kernel: some
// five divisions in a row took several hundred of the 14000 cycles of a single-token call (8.3
// us, 7.9 so).  The tile kernel gains nothing by them.
struct RowAt {
  int token, head;
};
__device__ __forceinline__ RowAt row_at(const ChunkParams& p, int packed) {
  const int t = div_page(packed, p.G, p.g_div);
  return {t, packed - t * p.G};
}
__device__ __forceinline__ int token_at(const ChunkParams& p, int packed) { return div_page(packed, p.G, p.g_div); }
__device__ __forceinline__ int div_s(const ChunkParams& p, int x) { return div_page(x, p.S, p.s_div); }
__device__ __forceinline__ int div_parts(const ChunkParams& p, int x) { return div_page(x, p.parts, p.parts_div); }
__device__ __forceinline__ int div_hkv(const ChunkParams& p, int x) { return div_page(x, p.Hkv, p.hkv_div); }

// One request's new tokens, checked against the plan.
struct ChunkRequest {
  int row0;  // first row of q
  int n;     // new tokens (at most max_q)
  int kv;    // positions, new tokens included
  bool bad;  // something was clamped
};

__device__ __forceinline__ ChunkRequest chunk_request(const ChunkParams& p, int b) {
  const int a0 = p.cu_q[b], a1 = p.cu_q[b + 1], len = p.kv_len[b];
  ChunkRequest r;
  r.row0 = min(max(a0, 0), p.total_q);
  const int end = min(max(a1, r.row0), p.total_q);
  r.n = min(end - r.row0, p.max_q);
  r.kv = min(max(len, 0), p.max_kv_len);
  r.bad = r.row0 != a0 || r.row0 + r.n != a1 || r.kv != len;
  return r;
}

// The positions that new tokens [ia, ib] of a request see together, as one
// axis of virtual tokens 0 .. U-1: the visible sinks first, then the window's
// run without a gap (virtual token v < sk is position v, any other position
// v + skip).  Packing the sinks in front of the window costs no tile of its
// own, and every virtual token is seen by some row.
struct ChunkSpan {
  int U, sk, skip;
  __device__ __forceinline__ int position(int v) const { return v < sk ? v : v + skip; }
};

// TREE: the new tokens are a tree's nodes, which all stand behind the context whatever the
// order that they are stored in: the context from the root's window on, and all nodes.
template <bool TREE = false>
__device__ __forceinline__ ChunkSpan chunk_span(const ChunkParams& p, const ChunkRequest& r, int ia, int ib) {
  ChunkSpan s = {0, 0, 0};
  if (TREE) {
    const int base = max(r.kv - r.n, 0);
    if (p.window > 0) {
      s.sk = min(p.sinks, base);
      s.skip = max(max(0, base - p.window + 1) - s.sk, 0);
    }
    s.U = r.kv - s.skip;
    return s;
  }
  const int first = r.kv - r.n + ia;
  const int hi = max(r.kv - r.n + ib + 1, 0);
  if (p.window > 0) {
    const int lo = max(0, first - p.window + 1);
    s.sk = min(p.sinks, hi);
    s.skip = max(lo - s.sk, 0);
  }
  s.U = hi - s.skip;
  return s;
}

// 2^x for a whole x <= 0 (0 below the normal range; NaN, from infinite maxima, stays NaN).
__device__ __forceinline__ float exp2_whole(float x) {
  if (x != x) return x;
  return x < -126.f ? 0.f : __int_as_float(((int)x + 127) << 23);
}

// 2^(m - M), the weight of a partition that saw something in the joint sum
// (whole maxima): never 0, so that an infinite numerator of a far smaller
// partition stays infinite (0 * inf would not).
__device__ __forceinline__ float part_weight(float m, float M) {
  return m == M ? 1.f : exp2_whole(fmaxf(m - M, -120.f));
}

// The sum that a partition leaves for a row, as the join reads it.  +0: the partition was
// empty and its numerators were not written.  -0: they were, by positions whose logits are
// all -inf; they are 0, or not finite where such a position has a non-finite V code.
__device__ __forceinline__ float part_sum(float l) { return l == 0.f ? -0.f : l; }
__device__ __forceinline__ bool part_written(float2 ml) { return __float_as_uint(ml.y) != 0u; }

// What one row sees on that axis: v < hi and (v >= lo or v < sk).
struct ChunkRow {
  int hi, lo;
  __device__ __forceinline__ bool sees(int v, int sk) const { return v < hi && (v >= lo || v < sk); }
};
// ... and a tree's row: of the context (v < hi) the same, of the nodes (v >= hi: node v - hi)
// those of its mask.  (Node numbers stay below the request's nodes: v < U.)
struct TreeRow {
  int hi, lo;
  const uint32_t* mask;
  __device__ __forceinline__ bool sees(int v, int sk) const {
    if (v < hi) return v >= lo || v < sk;
    const int j = v - hi;
    return (__ldg(mask + (j >> 5)) >> (j & 31)) & 1u;
  }
};
template <bool TREE>
struct RowOfTree {
  using type = ChunkRow;
};
template <>
struct RowOfTree<true> {
  using type = TreeRow;
};

// A row that sees everything (rows past the last one, whose results are dropped).
template <bool TREE>
__device__ __forceinline__ typename RowOfTree<TREE>::type any_row(int lo) {
  if constexpr (TREE)
    return {INT_MAX, lo, nullptr};
  else
    return {INT_MAX, lo};
}

template <bool TREE = false>
__device__ __forceinline__ typename RowOfTree<TREE>::type chunk_row(const ChunkParams& p, const ChunkRequest& r,
                                                                    const ChunkSpan& s, int i) {
  if constexpr (TREE) {
    TreeRow c;
    c.hi = r.kv - r.n - s.skip;
    c.lo = -s.skip;
    c.mask = p.mask + (int64_t)(r.row0 + i) * p.mask_stride;
    if (p.window > 0) {
      const int d = __ldg(p.depth + r.row0 + i), at = min(max(d, 0), r.n - 1);
      if (at != d) set_status(p.status, FP8KV_STATUS_BAD_LEN);
      c.lo = max(r.kv - r.n + at - p.window + 1, 0) - s.skip;
    }
    return c;
  } else {
    const int pos = r.kv - r.n + i;
    ChunkRow c;
    c.hi = pos + 1 - s.skip;
    c.lo = (p.window > 0 ? max(pos - p.window + 1, 0) : 0) - s.skip;
    return c;
  }
}

// Tiles of a partition where CTAs find their shares (share_of), from the length T for requests of two
// row tiles.
template <bool TREE>
__device__ __forceinline__ int share_tiles(int T, bool light) {
  return TREE && light ? (5 * T + 3) / 4 : T;
}

// Physical place of a position: false when its block is out of range.
__device__ __forceinline__ bool chunk_place(const ChunkParams& p, int b, int pos, int64_t& blk, int& slot) {
  const int page = div_page(pos, p.page_size, p.page_div);
  slot = pos - page * p.page_size;
  blk = p.block_table[(int64_t)b * p.bt_stride + page];
  return blk >= 0 && blk < p.num_kv_blocks;
}

// Exact FP8 -> fp16 for four bytes (byte pairs 0,1 and 2,3).
template <int FMT>
__device__ __forceinline__ void fp8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == FP8KV_KV_E5M2)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e5m2x2 %0, a;\n\tcvt.rn.f16x2.e5m2x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  else
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two floats rounded to the output type.
template <int DT>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
  if (DT == FP8KV_DTYPE_F16) return pack_half2(lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// bf16 query row -> fp16: the power of two that brings the row's largest
// magnitude (given as the bits of a non-negative float) to [2^14, 2^15), and
// its inverse.  Every element above 2^-28 of the largest is then an fp16
// normal, so the product is exact; a zero row, or one with infinities or
// NaNs, is left unscaled (its logits are 0, or not finite, either way).
struct RowScale {
  float to_f16, back;
};
__device__ __forceinline__ RowScale row_scale_bf16(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23);  // biased exponent (0: zero or subnormal)
  if (e == 255 || amax == 0.f) return {1.f, 1.f};
  const int k = min(14 - (e - 127), 126);            // power, kept representable with its inverse
  return {__uint_as_float((uint32_t)(127 + k) << 23), __uint_as_float((uint32_t)(127 - k) << 23)};
}

// Kind of a non-finite code, as bits: 1 NaN, 2 +inf, 4 -inf, 0 finite.
template <int FMT>
__device__ __forceinline__ uint32_t nonfinite_kind(uint32_t byte) {
  if (FMT == FP8KV_KV_E5M2) {
    if ((byte & 0x7Cu) != 0x7Cu) return 0u;
    return (byte & 3u) ? 1u : ((byte & 0x80u) ? 4u : 2u);
  }
  return (byte & 0x7Fu) == 0x7Fu ? 1u : 0u;
}
__device__ __forceinline__ float nonfinite_value(uint32_t kinds) {
  return ((kinds & 1u) || (kinds & 6u) == 6u) ? __uint_as_float(0x7FC00000u)
                                              : ((kinds & 2u) ? INFINITY : -INFINITY);
}

// Non-finite V codes.  PV products run over every token of a tile, and a weight
// of 0 times NaN would reach rows that do not see the token; such codes
// therefore enter the product as 0, and a CTA that met one re-reads its V
// bytes: `kinds` (one byte per (row, column), RC x D, zeroed here) receives
// the non-finite codes of the tokens that each row sees.  Rare path; all
// threads of the CTA, between barriers.
template <int D, int FMT, class RowOf>
__device__ __noinline__ void mark_nonfinite_v(const ChunkParams& p, uint32_t* kinds, int b, int g, int u0, int u1,
                                              ChunkSpan span, int RC, RowOf row_of) {
  for (int x = threadIdx.x; x < RC * D / 4; x += blockDim.x) kinds[x] = 0u;
  __syncthreads();
  constexpr int kC = D / 16;
  for (int64_t x = threadIdx.x; x < (int64_t)(u1 - u0) * kC; x += blockDim.x) {
    const int v = u0 + (int)(x / kC), c = (int)(x % kC);
    int64_t blk;
    int slot;
    if (!chunk_place(p, b, span.position(v), blk, slot)) continue;
    const uint4 w = *reinterpret_cast<const uint4*>(p.v_cache + blk * p.vsb + slot * p.vst + g * p.vsh + c * 16);
    if (nonfinite_codes(w, FMT == FP8KV_KV_E5M2) == 0u) continue;
    const uint32_t wa[4] = {w.x, w.y, w.z, w.w};
    for (int j = 0; j < 16; ++j) {
      const uint32_t kind = nonfinite_kind<FMT>((wa[j / 4] >> (8 * (j % 4))) & 0xFFu);
      if (kind == 0u) continue;
      const int d = c * 16 + j;
      for (int i = 0; i < RC; ++i) {
        const auto row = row_of(i);
        if (row.sees(v, span.sk)) atomicOr(&kinds[i * (D / 4) + d / 4], kind << (8 * (d % 4)));
      }
    }
  }
  __syncthreads();
}

}  // namespace fp8kv
