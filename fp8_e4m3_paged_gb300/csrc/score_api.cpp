// C ABI entry points of the gathered weights: planning (host only), argument
// validation, dispatch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "args_check.h"
#include "fp8kv_attn.h"
#include "output_layout.h"
#include "score.h"

using namespace fp8kv;

namespace {
constexpr int64_t kScoreStreamBytes = 56 << 20;
constexpr int64_t kScoreLogitBytes = 4ll << 30;
}

extern "C" int fp8kv_attn_cache_score_plan(const fp8kv_chunk_desc* d, fp8kv_cache_score_plan_t* plan) {
  if (!d || !plan) return FP8KV_EINVAL;
  // the chunk attention's checks; its plan is not used further
  fp8kv_chunk_plan_t chunk;
  fp8kv_chunk_desc same = *d;
  same.kernel = FP8KV_CHUNK_AUTO;
  same.num_splits = 0;
  const int rc = fp8kv_attn_chunk_plan(&same, &chunk);
  if (rc != FP8KV_OK) return rc;
  if (d->num_splits < 0 || d->num_splits > 65535 || d->kernel < FP8KV_CHUNK_AUTO || d->kernel > FP8KV_CHUNK_TILE)
    return FP8KV_EINVAL;
  if (d->window > 0) return FP8KV_EUNSUPPORTED;
  const int64_t pairs = (int64_t)d->batch * d->num_kv_heads;
  if (pairs > 65535 || d->max_kv_len > (1 << 26)) return FP8KV_EUNSUPPORTED;  // grids

  fp8kv_cache_score_plan_t P;
  std::memset(&P, 0, sizeof(P));
  P.revision = FP8KV_ATTN_REVISION;
  P.batch = chunk.batch;
  P.total_q = chunk.total_q;
  P.max_q = chunk.max_q;
  P.num_q_heads = chunk.num_q_heads;
  P.num_kv_heads = chunk.num_kv_heads;
  P.head_dim = chunk.head_dim;
  P.page_size = chunk.page_size;
  P.max_kv_len = chunk.max_kv_len;
  P.max_blocks = chunk.max_blocks;
  P.num_kv_blocks = chunk.num_kv_blocks;
  P.dtype = chunk.dtype;
  P.kv_format = chunk.kv_format;
  P.group = chunk.group;
  P.num_sms = chunk.num_sms;
  const int64_t rows = (int64_t)P.max_q * P.group;  // query vectors per (request, KV head)
  const int64_t len = std::max(P.max_kv_len, 1), sms = P.num_sms;
  P.kernel = d->kernel;
  if (P.kernel == FP8KV_CHUNK_AUTO) {
    // Up to 16 query vectors stream K once.  More stream it anew for each 16 and keep all logits, which
    // pays while that is little, because the tile kernel's two passes take 20 us on the shortest contexts.
    // us, stream / tile, 8 KV heads x 4, D 128, by the bytes counted here: 32 tokens on 500 (8 MB) 9.8 / 18.5,
    // 4 x 500 (31 MB) 16.6 / 24.9, 4 x 1000 (63 MB) 27.0 / 26.3, 16 x 500 (125 MB) 44 / 28; 8 tokens on
    // 4 x 2000 (31 MB) 13.6 / 29.1, 16 x 1000 (66 MB) 20 / 37; 48 requests of 16 tokens on 20 (8 MB) 13 / 48.
    // The border is the one of 32 tokens.  Fewer still stream faster past it and do not: those 8, and 5 tokens
    // on 64 x 500 (108 MB) 35 / 80; 64 on 4 x 500 (74 MB) 42 / 31 are on the right side.
    const int64_t bytes = pairs * len * (8 * rows + ceil_div(rows, kScoreGroupRows) * P.head_dim);
    // (and the workspace stays in bounds: the tile kernel keeps no logits)
    const bool stream = pairs * len * score_vectors(rows) * 4 <= kScoreLogitBytes &&
                        (rows <= kScoreGroupRows || (rows <= kScoreStreamRows && bytes <= kScoreStreamBytes));
    P.kernel = stream ? FP8KV_CHUNK_STREAM : FP8KV_CHUNK_TILE;
  }
  if (P.kernel == FP8KV_CHUNK_STREAM && rows > kScoreStreamRows) return FP8KV_EUNSUPPORTED;
  P.partial_offset = 256;
  int64_t floats;
  if (P.kernel == FP8KV_CHUNK_STREAM) {
    // partitions of one length: some four CTAs per SM, of 128 to 2048 positions
    const int64_t row_groups = ceil_div(rows, kScoreGroupRows);
    int64_t part = std::min<int64_t>(2048, std::max<int64_t>(128, ceil_div(pairs * row_groups * len, 4 * sms)));
    if (d->num_splits) part = ceil_div(len, d->num_splits);
    // (a lane's FP32 sum has 1 of 32 positions; 2^26 positions are 1024 partitions at least)
    part = align_up(std::min<int64_t>(std::max(part, ceil_div(len, 65535)), 65536), 128);
    P.num_splits = (int32_t)ceil_div(len, part);
    P.vectors = score_vectors(rows);
    P.row_groups = 1;
    P.stat_part = P.col_part = (int32_t)part;
    floats = pairs * len * P.vectors;
  } else {
    const int64_t tile = P.head_dim == 256 ? 128 : 256, tiles = ceil_div(len, kChunkTileTokens);
    P.row_tiles = (int32_t)(P.total_q * (int64_t)P.group / tile + std::min(P.batch, P.total_q));
    const int64_t units = std::max<int64_t>((int64_t)P.row_tiles * P.num_kv_heads, 1);
    // rows' sums: some four CTAs per SM of at least 8 tiles, one per row block where those are many
    int64_t part = units >= 2 * sms ? tiles : std::min(tiles, std::max<int64_t>(8, ceil_div(units * tiles, 3 * sms)));
    if (d->num_splits) part = ceil_div(tiles, d->num_splits);
    part = std::max<int64_t>(part, ceil_div(tiles, 65535));
    P.stat_part = (int32_t)(part * kChunkTileTokens);
    P.num_splits = (int32_t)ceil_div(len, P.stat_part);
    // columns: likewise; several row tiles meet in shared memory, which holds 2048 positions
    const int64_t blocks = ceil_div(rows, tile);
    const int64_t most = rows > 128 ? kScoreAccTokens / kChunkTileTokens : tiles;
    part = std::min(most, std::max<int64_t>(8, ceil_div(pairs * tiles, 3 * sms)));
    part = std::max<int64_t>({part, 1, rows > 128 ? 1 : ceil_div(tiles, 65535)});  // (16 tiles are enough for 2^26)
    P.col_part = (int32_t)(part * kChunkTileTokens);
    const int64_t ctas = std::max<int64_t>(pairs * ceil_div(len, P.col_part), 1);
    P.row_groups = (int32_t)std::max<int64_t>(1, std::min({blocks, 6 * sms / ctas, (int64_t)64}));
    floats = P.row_groups > 1 ? P.row_groups * pairs * len : 0;
    // One row block per request, and CTAs enough for one wave: shares by the lengths on the device.
    const int64_t per_head = sms / P.num_kv_heads;
    if (d->num_splits == 0 && blocks <= 1 && per_head >= 1 && P.batch <= std::min<int64_t>(per_head, kShareMax)) {
      P.per_head = (int32_t)per_head;
      P.num_splits = (int32_t)std::min(tiles, per_head);
      P.row_groups = rows <= 128 ? 1 : 2;  // (two row tiles: each has its sums in the workspace)
      floats = P.row_groups > 1 ? P.row_groups * pairs * len : 0;
    }
  }
  if (P.num_splits > 65535 || (int64_t)P.row_tiles * P.num_kv_heads > 0x7fffffff) return FP8KV_EUNSUPPORTED;
  P.ml_offset = align_up(P.partial_offset + floats * 4, 256);
  P.workspace_bytes = align_up(P.ml_offset + (int64_t)P.num_splits * P.total_q * P.num_q_heads * 8, 256);
  *plan = P;
  return FP8KV_OK;
}

extern "C" int fp8kv_attn_cache_score(const fp8kv_cache_score_plan_t* plan, const fp8kv_cache_score_args* a,
                                      fp8kv_stream_t stream) {
  if (!plan || !a) return FP8KV_EINVAL;
  if (plan->revision != FP8KV_ATTN_REVISION) return FP8KV_EVERSION;
  if (plan->kernel != FP8KV_CHUNK_STREAM && plan->kernel != FP8KV_CHUNK_TILE) return FP8KV_EINVAL;
  if (plan->num_splits < 1 || plan->row_groups < 1 || plan->group < 1 || plan->page_size < 1 ||
      plan->num_kv_heads < 1 || plan->stat_part < 1 || plan->col_part < 1 || !fp8_format(plan->kv_format) ||
      (plan->dtype != FP8KV_DTYPE_F16 && plan->dtype != FP8KV_DTYPE_BF16))
    return FP8KV_EINVAL;
  if (!a->workspace || !aligned(a->workspace, 256)) return FP8KV_EINVAL;
  if ((int64_t)a->workspace_bytes < plan->workspace_bytes) return FP8KV_EWORKSPACE;
  if (plan->batch == 0 || plan->total_q == 0 || plan->max_kv_len == 0) return FP8KV_OK;
  if (!a->q || !a->k_cache || !aligned(a->q, 16) || !aligned(a->k_cache, 16)) return FP8KV_EINVAL;
  const int64_t es[] = {a->q_stride_token, a->q_stride_head};
  const int64_t bs[] = {a->k_stride_block, a->k_stride_token, a->k_stride_head};
  const int64_t fs[] = {a->score_in_stride_req, a->score_in_stride_head, a->score_stride_req, a->score_stride_head};
  if (!strides_ok(es, 2, 8) || !strides_ok(bs, 3, 16) || !strides_ok(fs, 4, 1)) return FP8KV_EINVAL;
  if (!a->cu_q || !a->kv_len || !aligned(a->cu_q, 4) || !aligned(a->kv_len, 4)) return FP8KV_EINVAL;
  if (!a->block_table || !aligned(a->block_table, 4) || a->block_table_stride < plan->max_blocks) return FP8KV_EINVAL;
  if (!std::isfinite(a->softmax_scale) || !std::isfinite(a->decay) || !aligned(a->k_scale_dev, 4) ||
      (!a->k_scale_dev && !std::isfinite(a->k_scale)))
    return FP8KV_EINVAL;
  if (!a->score || !aligned(a->score, 4) || !aligned(a->score_in, 4)) return FP8KV_EINVAL;
  if (!apart(plan->batch, fs[2], plan->num_kv_heads, fs[3], plan->max_kv_len)) return FP8KV_EINVAL;
  // The same buffer is read and written element by element; others, in no order, share no place.
  if (a->score_in == a->score ? fs[0] != fs[2] || fs[1] != fs[3]
                              : a->score_in && meet({plan->batch, fs[0], plan->num_kv_heads, fs[1]},
                                                    {plan->batch, fs[2], plan->num_kv_heads, fs[3]}, plan->max_kv_len,
                                                    floats_between(a->score_in, a->score)))
    return FP8KV_EINVAL;

  ScoreParams p;
  std::memset(&p, 0, sizeof(p));
  ChunkParams& c = p.c;
  c.B = plan->batch;
  c.total_q = plan->total_q;
  c.max_q = plan->max_q;
  c.Hq = plan->num_q_heads;
  c.Hkv = plan->num_kv_heads;
  c.G = plan->group;
  c.S = plan->num_splits;
  c.page_size = plan->page_size;
  auto inverse = [](int32_t n) { return n >= 2 ? ~0ull / (uint64_t)n + 1 : 0ull; };
  c.page_div = inverse(plan->page_size);
  c.g_div = inverse(plan->group);
  c.s_div = inverse(plan->num_splits);
  c.hkv_div = inverse(plan->num_kv_heads);
  c.max_kv_len = plan->max_kv_len;
  c.num_kv_blocks = plan->num_kv_blocks;
  c.row_tiles = plan->row_tiles;
  c.q = reinterpret_cast<const uint16_t*>(a->q);
  c.q_st = a->q_stride_token;
  c.q_sh = a->q_stride_head;
  c.k_cache = a->k_cache;
  c.ksb = bs[0];
  c.kst = bs[1];
  c.ksh = bs[2];
  c.block_table = a->block_table;
  c.bt_stride = a->block_table_stride;
  c.cu_q = a->cu_q;
  c.kv_len = a->kv_len;
  c.softmax_scale = a->softmax_scale;
  c.k_scale = a->k_scale;
  c.k_scale_dev = a->k_scale_dev;
  char* ws = reinterpret_cast<char*>(a->workspace);
  c.status = reinterpret_cast<unsigned int*>(ws);
  c.ml = reinterpret_cast<float2*>(ws + plan->ml_offset);
  p.stat_part = plan->stat_part;
  p.col_part = plan->col_part;
  p.groups = plan->row_groups;
  p.per_head = plan->per_head;
  p.vectors = plan->vectors;
  p.logits = p.partial = reinterpret_cast<float*>(ws + plan->partial_offset);
  p.in = a->score_in;
  p.in_sr = fs[0];
  p.in_sh = fs[1];
  p.decay = a->decay;
  p.out = a->score;
  p.out_sr = fs[2];
  p.out_sh = fs[3];
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return done(plan->kernel == FP8KV_CHUNK_STREAM ? launch_score_stream(plan, p, st) : launch_score_tile(plan, p, st));
}
