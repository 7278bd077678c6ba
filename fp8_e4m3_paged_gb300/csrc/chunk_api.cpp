// C ABI entry points of the chunk attention, the cache read and the scale
// calibration: planning (host only), argument validation, dispatch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "args_check.h"
#include "chunk.h"
#include "fp8kv_attn.h"
#include "output_layout.h"

using namespace fp8kv;

namespace {

int make_plan(const fp8kv_chunk_desc* d, fp8kv_chunk_plan_t* plan, bool tree) {
  if (!d || !plan) return FP8KV_EINVAL;
  if (d->batch < 0 || d->total_q < 0 || d->max_q < 1 || d->num_q_heads < 1 || d->num_kv_heads < 1)
    return FP8KV_EINVAL;
  if (d->num_q_heads % d->num_kv_heads) return FP8KV_EINVAL;
  if (d->page_size < 1 || d->max_kv_len < 0 || d->max_blocks < 0 || d->num_kv_blocks < 1) return FP8KV_EINVAL;
  if ((int64_t)d->max_blocks * d->page_size < d->max_kv_len) return FP8KV_EINVAL;
  if (d->window < 0 || d->sinks < 0 || (d->window == 0 && d->sinks > 0)) return FP8KV_EINVAL;
  if (d->dtype != FP8KV_DTYPE_F16 && d->dtype != FP8KV_DTYPE_BF16) return FP8KV_EINVAL;
  if (d->num_sms < 0 || d->num_splits < 0 || d->num_splits > 65535) return FP8KV_EINVAL;
  if (d->kernel < FP8KV_CHUNK_AUTO || d->kernel > FP8KV_CHUNK_TILE) return FP8KV_EINVAL;
  if (d->kv_format == FP8KV_KV_BF16) return FP8KV_EUNSUPPORTED;
  if (!fp8_format(d->kv_format)) return FP8KV_EINVAL;
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return FP8KV_EUNSUPPORTED;
  // no request has more new tokens than there are rows
  const int32_t max_q = std::min(d->max_q, std::max(d->total_q, 1));
  // 32-bit positions, packed rows and grid sizes
  const int64_t group = d->num_q_heads / d->num_kv_heads;
  if (d->total_q > (1 << 30) || d->max_q > (1 << 24) || d->max_kv_len > (1 << 30) || d->num_kv_heads > 65535 ||
      max_q * group > (1 << 30) || (int64_t)d->total_q * d->num_q_heads > ((int64_t)1 << 32) ||
      d->num_sms > 65535)
    return FP8KV_EUNSUPPORTED;
  if (tree && max_q > kTreeNodesMax) return FP8KV_EUNSUPPORTED;
  if (d->kernel == FP8KV_CHUNK_STREAM && max_q * group > 65535 * (int64_t)kChunkStreamRows)
    return FP8KV_EUNSUPPORTED;

  int sms = d->num_sms;
  if (sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FP8KV_ECUDA;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return FP8KV_ECUDA;
    if (sms < 1) return FP8KV_ECUDA;
  }

  fp8kv_chunk_plan_t P;
  std::memset(&P, 0, sizeof(P));
  P.revision = FP8KV_ATTN_REVISION;
  P.batch = d->batch;
  P.total_q = d->total_q;
  P.max_q = max_q;
  P.num_q_heads = d->num_q_heads;
  P.num_kv_heads = d->num_kv_heads;
  P.head_dim = d->head_dim;
  P.page_size = d->page_size;
  P.max_kv_len = d->max_kv_len;
  P.max_blocks = d->max_blocks;
  P.num_kv_blocks = d->num_kv_blocks;
  // a window that reaches back over every context is none
  P.window = d->window >= d->max_kv_len ? 0 : d->window;
  P.sinks = P.window ? std::min(d->sinks, d->max_kv_len) : 0;
  P.dtype = d->dtype;
  P.kv_format = d->kv_format;
  P.tree = tree;
  P.group = (int32_t)group;
  P.num_sms = sms;

  const int64_t rows = P.max_q * group;  // query vectors per (request, KV head)
  const int64_t pairs = (int64_t)P.batch * P.num_kv_heads;  // the stream kernel's grid.x
  const int64_t stream_units = std::min<int64_t>(pairs, 1ll << 32) * ceil_div(rows, kChunkStreamRows);
  auto seen_by = [&](int64_t tokens) -> int64_t {  // positions that so many tokens see together, at most
    return P.window ? std::min<int64_t>(P.max_kv_len, (int64_t)P.window + P.sinks + tokens - 1) : P.max_kv_len;
  };
  P.kernel = d->kernel;
  if (P.kernel == FP8KV_CHUNK_AUTO) {
    // The stream kernel takes 16 query vectors at a time and reads the positions
    // anew for the next 16; the tile kernel serves 256 (128) from one read, but
    // starts slower and leaves SMs idle where there are few tiles.  So more
    // than 16 vectors stream while the positions are few (`units`: CTAs of the
    // stream kernel before the context is split; us, stream / tile):
    //   units few, any number of vectors: 32 units x 2064 positions 13.9 / 15.6, 24 x 340 (D 64)
    //   6.9 / 12.1, 26 x 400 (D 256) 13.1 / 16.6, 16 x 2008 12.6 / 13.6, but 16 x 4008 17.0 / 15.5;
    //   up to 32 vectors: 64 units x 1008 12.7 / 15.1, x 2008 17.2 / 18.3, 256 x 308 13.2 / 13.8,
    //   but 256 x 2008 54.7 / 38.6, 512 x 8008 309 / 249.
    const int64_t seen = seen_by(P.max_q);
    const bool few = 2 * stream_units <= sms || (rows <= 32 && (stream_units <= sms || seen <= 512));
    const bool stream = rows <= kChunkStreamRows || (seen * P.head_dim <= 5 << 16 && few);
    P.kernel = stream ? FP8KV_CHUNK_STREAM : FP8KV_CHUNK_TILE;
  }

  // Partitions: about one CTA per slot of the GPU, none shorter than `unit`
  // positions of what one CTA's rows see together.
  // Stream kernel: more than two CTAs per SM only where each keeps 512
  // positions (us, with / without that: 128 units x 300 positions S = 2 8.4, S = 4 9.8;
  // 256 x 500 S = 1 11.9, S = 2 12.4; 64 x 1000 S = 4 9.1, S = 8 10.0; and 256 x 2000 S = 2 32.5,
  // S = 1 35.4).
  int64_t units, slots, unit, span_q;
  if (P.kernel == FP8KV_CHUNK_STREAM) {
    units = stream_units;
    slots = (int64_t)sms * (P.head_dim == 64 ? 5 : P.head_dim == 128 ? 4 : 2);
    unit = 4 * kChunkStreamBlock;
    span_q = P.max_q;
  } else {
    const int64_t tile = chunk_tile_rows(P.head_dim);
    P.row_tiles = (int32_t)(P.total_q * group / tile + std::min(P.batch, P.total_q));
    units = (int64_t)P.row_tiles * P.num_kv_heads;
    slots = sms;
    unit = kChunkTileTokens;
    span_q = tree ? P.max_q : std::min<int64_t>(P.max_q, ceil_div(tile, group) + 1);
  }
  const int64_t seen = seen_by(span_q);
  int64_t S = units ? slots / units : 1;
  S = std::min(S, ceil_div(seen, unit));
  if (P.kernel == FP8KV_CHUNK_STREAM) {
    if (units) S = std::max(std::min(2 * sms / units, ceil_div(seen, unit)), std::min(slots / units, seen / 512));
    if (S > kChunkClusterMax && seen <= kChunkClusterMax * 8 * unit) S = kChunkClusterMax;
  } else {
    // The CTAs of one request are equally long, so the last of their waves is
    // worth filling: the S whose waves times a CTA's time (its positions, and
    // about 900 more for its start and end) is least.  8 KV heads x 2048 tokens x 4
    // on 30000 positions, 152 SMs: S = 1 (2 waves) 897 us, 2 (4) 929, 3 (6) 937, 4 (7)
    // 861, 5 (9) 899, 7 (12) 902.  (CTAs of several requests differ in length and fill
    // the gaps themselves: 16 requests, 41 row tiles x 8 heads, S = 1: 133 us, 2: 164, 4: 192.)
    if (P.batch == 1) {
      const int64_t ctas = ceil_div(rows, chunk_tile_rows(P.head_dim)) * P.num_kv_heads;
      // (a tree's CTAs are all equally long and few: up to one wave of them)
      const int64_t most = std::min(std::max<int64_t>(8, tree ? sms / ctas : S), ceil_div(seen, unit));
      int64_t best = INT64_MAX;
      for (int64_t n = 1; n <= most; ++n) {
        const int64_t cost = ceil_div(ctas * n, sms) * (ceil_div(seen, n) + 900);
        if (cost < best) {
          best = cost;
          S = n;
        }
      }
    }
  }
  if (d->num_splits) S = d->num_splits;
  S = std::min<int64_t>(std::max<int64_t>(1, S), 65535);
  P.min_splits = (int32_t)S;
  // No FP32 sum over more than kChunkMaxSum positions, whoever chose the partitions: the
  // kernels use the further ones for contexts that need them.  (64 decodes of 4000 positions,
  // planned for 4000: 93 us; planned for 2^20: 102, and 162 were all 16 partitions used.)
  P.max_part = (int32_t)chunk_max_part(P.kernel);
  if (tree && P.kernel == FP8KV_CHUNK_TILE && P.batch > 1 && d->num_splits == 0) {
    // Trees of several requests, a CTA for each row block and KV head: the longest of 16 contexts of 100 to
    // 8000 positions took 140 of 143 us.  One row block per request: shares by the lengths on the device, of a
    // wave of CTAs and half as many more as there are requests, whose last partitions are
    // short (that batch in us with none more 89, half 76, as many 83; partitions of one length chosen here 82).
    // Else partitions of one length, so that a long context becomes as many CTAs as it takes.
    const int64_t tiles = ceil_div(seen, unit), per_head = sms / P.num_kv_heads + (P.batch - 1) / 2;
    // (the longest share that the lengths can lead to, lengthened for requests of one row tile)
    const int64_t longest = per_head > P.batch ? ceil_div(seen * P.batch, per_head - P.batch) : seen;
    if (rows <= chunk_tile_rows(P.head_dim) && P.batch <= std::min<int64_t>(per_head, kShareMax) &&
        std::min(seen, 2 * longest + 2 * unit) <= P.max_part) {
      P.per_head = (int32_t)per_head;
      S = std::max<int64_t>(1, std::min(tiles, per_head));
      P.min_splits = (int32_t)S;
    } else {
      const int64_t part = std::min<int64_t>(32, std::max<int64_t>(8, units * tiles / (8 * sms)));
      P.max_part = (int32_t)std::min<int64_t>(P.max_part, part * unit);
      P.min_splits = 1;
    }
  }
  if (P.per_head == 0) S = std::max(S, ceil_div(seen, P.max_part));
  // grid.x
  if ((P.kernel == FP8KV_CHUNK_STREAM ? pairs : (int64_t)P.row_tiles * P.num_kv_heads) > 0x7fffffff)
    return FP8KV_EUNSUPPORTED;
  P.num_splits = (int32_t)S;

  const int64_t nvec = S > 1 && !chunk_clustered(&P) ? S * P.total_q * P.num_q_heads : 0;
  P.partial_offset = 256;
  P.ml_offset = align_up(P.partial_offset + nvec * P.head_dim * 4, 256);
  P.workspace_bytes = align_up(P.ml_offset + nvec * 8, 256);
  *plan = P;
  return FP8KV_OK;
}

int build_chunk(const fp8kv_chunk_plan_t* plan, const fp8kv_chunk_args* a, ChunkParams* p) {
  if (!plan || !a) return FP8KV_EINVAL;
  if (plan->revision != FP8KV_ATTN_REVISION) return FP8KV_EVERSION;
  std::memset(p, 0, sizeof(*p));
  if (plan->kernel != FP8KV_CHUNK_STREAM && plan->kernel != FP8KV_CHUNK_TILE) return FP8KV_EINVAL;
  if (plan->num_splits < 1 || plan->min_splits < 1 || plan->min_splits > plan->num_splits || plan->max_part < 1 ||
      plan->group < 1 || plan->page_size < 1 || !fp8_format(plan->kv_format) ||
      (plan->dtype != FP8KV_DTYPE_F16 && plan->dtype != FP8KV_DTYPE_BF16))
    return FP8KV_EINVAL;
  if (!a->workspace || !aligned(a->workspace, 256)) return FP8KV_EINVAL;
  if ((int64_t)a->workspace_bytes < plan->workspace_bytes) return FP8KV_EWORKSPACE;
  if (plan->batch == 0 || plan->total_q == 0) return FP8KV_OK;
  const void* ptrs[] = {a->q, a->out, a->k_cache, a->v_cache};
  for (const void* x : ptrs)
    if (!x || !aligned(x, 16)) return FP8KV_EINVAL;
  const int64_t es[] = {a->q_stride_token, a->q_stride_head, a->out_stride_token, a->out_stride_head};
  const int64_t bs[] = {a->k_stride_block, a->k_stride_token, a->k_stride_head,
                        a->v_stride_block, a->v_stride_token, a->v_stride_head};
  if (!strides_ok(es, 4, 8) || !strides_ok(bs, 6, 16)) return FP8KV_EINVAL;
  if (!apart(plan->total_q, es[2], plan->num_q_heads, es[3], plan->head_dim)) return FP8KV_EINVAL;
  if (!a->cu_q || !a->kv_len || !aligned(a->cu_q, 4) || !aligned(a->kv_len, 4)) return FP8KV_EINVAL;
  if (plan->max_kv_len > 0 && (!a->block_table || !aligned(a->block_table, 4))) return FP8KV_EINVAL;
  if (a->block_table_stride < plan->max_blocks) return FP8KV_EINVAL;
  if (!std::isfinite(a->softmax_scale)) return FP8KV_EINVAL;
  if (!scales_ok(*a)) return FP8KV_EINVAL;

  p->B = plan->batch;
  p->total_q = plan->total_q;
  p->max_q = plan->max_q;
  p->Hq = plan->num_q_heads;
  p->Hkv = plan->num_kv_heads;
  p->G = plan->group;
  p->S = plan->num_splits;
  p->parts = plan->min_splits;
  p->max_part = plan->max_part;
  p->per_head = plan->per_head;
  p->page_size = plan->page_size;
  auto inverse = [](int32_t n) { return n >= 2 ? ~0ull / (uint64_t)n + 1 : 0ull; };
  p->page_div = inverse(plan->page_size);
  p->g_div = inverse(plan->group);
  p->s_div = inverse(plan->num_splits);
  p->parts_div = inverse(plan->min_splits);
  p->hkv_div = inverse(plan->num_kv_heads);
  p->max_kv_len = plan->max_kv_len;
  p->num_kv_blocks = plan->num_kv_blocks;
  p->window = plan->window;
  p->sinks = plan->sinks;
  p->row_tiles = plan->row_tiles;
  p->q = reinterpret_cast<const uint16_t*>(a->q);
  p->q_st = a->q_stride_token;
  p->q_sh = a->q_stride_head;
  p->out = reinterpret_cast<uint16_t*>(a->out);
  p->o_st = a->out_stride_token;
  p->o_sh = a->out_stride_head;
  p->k_cache = a->k_cache;
  p->v_cache = a->v_cache;
  p->ksb = bs[0];
  p->kst = bs[1];
  p->ksh = bs[2];
  p->vsb = bs[3];
  p->vst = bs[4];
  p->vsh = bs[5];
  p->block_table = a->block_table;
  p->bt_stride = a->block_table_stride;
  p->cu_q = a->cu_q;
  p->kv_len = a->kv_len;
  p->softmax_scale = a->softmax_scale;
  p->k_scale = a->k_scale;
  p->v_scale = a->v_scale;
  p->k_scale_dev = a->k_scale_dev;
  p->v_scale_dev = a->v_scale_dev;
  char* ws = reinterpret_cast<char*>(a->workspace);
  p->status = reinterpret_cast<unsigned int*>(ws);
  p->share = reinterpret_cast<int32_t*>(ws) + 1;
  p->partial = reinterpret_cast<float*>(ws + plan->partial_offset);
  p->ml = reinterpret_cast<float2*>(ws + plan->ml_offset);
  return FP8KV_OK;
}

}  // namespace

extern "C" int fp8kv_attn_chunk_plan(const fp8kv_chunk_desc* d, fp8kv_chunk_plan_t* plan) {
  return make_plan(d, plan, false);
}

extern "C" int fp8kv_attn_tree_plan(const fp8kv_chunk_desc* d, fp8kv_chunk_plan_t* plan) {
  return make_plan(d, plan, true);
}

extern "C" int fp8kv_attn_chunk(const fp8kv_chunk_plan_t* plan, const fp8kv_chunk_args* a, fp8kv_stream_t stream) {
  ChunkParams p;
  const int rc = build_chunk(plan, a, &p);
  if (rc != FP8KV_OK) return rc;
  if (plan->tree) return FP8KV_EINVAL;  // (causal rows: not what the plan is for)
  if (plan->batch == 0 || plan->total_q == 0) return FP8KV_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e =
      plan->kernel == FP8KV_CHUNK_STREAM ? launch_chunk_stream(plan, p, st) : launch_chunk_tile(plan, p, st);
  if (e == cudaSuccess && p.S > 1 && !chunk_clustered(plan)) e = launch_chunk_join(plan, p, st);
  return done(e);
}

extern "C" int fp8kv_attn_tree(const fp8kv_chunk_plan_t* plan, const fp8kv_tree_args* a, fp8kv_stream_t stream) {
  ChunkParams p;
  const int rc = build_chunk(plan, a ? &a->chunk : nullptr, &p);
  if (rc != FP8KV_OK) return rc;
  if (!plan->tree || plan->max_q > kTreeNodesMax) return FP8KV_EINVAL;
  if (plan->batch == 0 || plan->total_q == 0) return FP8KV_OK;
  if (!a->mask || !aligned(a->mask, 4) || a->mask_stride < ceil_div(plan->max_q, 32)) return FP8KV_EINVAL;
  if (plan->window > 0 && (!a->depth || !aligned(a->depth, 4))) return FP8KV_EINVAL;
  p.mask = a->mask;
  p.mask_stride = a->mask_stride;
  p.depth = a->depth;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = plan->kernel == FP8KV_CHUNK_STREAM ? launch_tree_stream(plan, p, st) : launch_tree_tile(plan, p, st);
  if (e == cudaSuccess && p.S > 1 && !chunk_clustered(plan)) e = launch_tree_join(plan, p, st);
  return done(e);
}

extern "C" int fp8kv_attn_cache_read(const fp8kv_cache_read_args* a, fp8kv_stream_t stream) {
  if (!a) return FP8KV_EINVAL;
  if (a->batch < 0 || a->total < 0 || a->num_kv_heads < 1 || a->page_size < 1 || a->max_blocks < 1 ||
      a->num_kv_blocks < 1)
    return FP8KV_EINVAL;
  if (a->head_dim < 16 || a->head_dim > 1024 || a->head_dim % 16) return FP8KV_EINVAL;
  if (a->num_kv_heads > 65535) return FP8KV_EUNSUPPORTED;  // 32-bit places within a row
  if (a->dtype != FP8KV_DTYPE_F16 && a->dtype != FP8KV_DTYPE_BF16 && a->dtype != FP8KV_DTYPE_F32)
    return FP8KV_EINVAL;
  if (!fp8_format(a->kv_format)) return FP8KV_EINVAL;
  if (a->batch == 0 || a->total == 0) return FP8KV_OK;
  const void* ptrs[] = {a->k_cache, a->v_cache, a->k_out, a->v_out};
  for (const void* x : ptrs)
    if (!x || !aligned(x, 16)) return FP8KV_EINVAL;
  const int64_t es[] = {a->ko_stride_token, a->ko_stride_head, a->vo_stride_token, a->vo_stride_head};
  const int64_t bs[] = {a->kc_stride_block, a->kc_stride_token, a->kc_stride_head,
                        a->vc_stride_block, a->vc_stride_token, a->vc_stride_head};
  if (!strides_ok(es, 4, 8) || !strides_ok(bs, 6, 16)) return FP8KV_EINVAL;
  if (!apart(a->total, es[0], a->num_kv_heads, es[1], a->head_dim) ||
      !apart(a->total, es[2], a->num_kv_heads, es[3], a->head_dim))
    return FP8KV_EINVAL;
  if (!a->block_table || !a->cu_len || a->block_table_stride < a->max_blocks) return FP8KV_EINVAL;
  if (!aligned(a->block_table, 4) || !aligned(a->cu_len, 4) || !aligned(a->start, 4) || !aligned(a->status, 4))
    return FP8KV_EINVAL;
  if (!scales_ok(*a)) return FP8KV_EINVAL;
  return done(launch_cache_read(*a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int fp8kv_attn_cache_calibrate(const fp8kv_calibrate_args* a, fp8kv_stream_t stream) {
  if (!a) return FP8KV_EINVAL;
  if (a->num_tokens < 0 || a->num_kv_heads < 1) return FP8KV_EINVAL;
  if (a->head_dim < 16 || a->head_dim > 1024 || a->head_dim % 16) return FP8KV_EINVAL;
  if (a->num_kv_heads > 65535) return FP8KV_EUNSUPPORTED;  // 32-bit places within a row
  if (a->dtype != FP8KV_DTYPE_F16 && a->dtype != FP8KV_DTYPE_BF16) return FP8KV_EINVAL;
  if (!fp8_format(a->kv_format)) return FP8KV_EINVAL;
  if (a->num_tokens == 0) return FP8KV_OK;
  if (!a->k || !a->v || !aligned(a->k, 16) || !aligned(a->v, 16)) return FP8KV_EINVAL;
  const int64_t es[] = {a->k_stride_token, a->k_stride_head, a->v_stride_token, a->v_stride_head};
  if (!strides_ok(es, 4, 8) || !aligned(a->slot_mapping, 8)) return FP8KV_EINVAL;
  if (!a->k_scale || !a->v_scale || a->k_scale == a->v_scale || !aligned(a->k_scale, 4) || !aligned(a->v_scale, 4))
    return FP8KV_EINVAL;
  return done(launch_calibrate(*a, reinterpret_cast<cudaStream_t>(stream)));
}
