// C ABI entry points of the selection and the move of cached positions:
// argument validation, dispatch.
#include <cstdint>

#include <cuda_runtime.h>

#include "args_check.h"
#include "evict.h"
#include "fp8kv_attn.h"
#include "output_layout.h"

using namespace fp8kv;

namespace {

// SMs of the current device (0: the call failed).
int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Whether two arrays of n int32 share bytes.
bool overlap(const int32_t* x, const int32_t* y, int64_t n) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(x), q = reinterpret_cast<uintptr_t>(y);
  return (p < q ? q - p : p - q) < (uintptr_t)(4 * n);
}

}  // namespace

extern "C" int fp8kv_attn_cache_select(const fp8kv_cache_select_args* a, fp8kv_stream_t stream) {
  if (!a) return FP8KV_EINVAL;
  if (a->batch < 0 || a->num_kv_heads < 1 || a->max_len < 0 || a->budget < 1 || a->sinks < 0 || a->recent < 0)
    return FP8KV_EINVAL;
  if (a->lists != 1 && a->lists != a->num_kv_heads) return FP8KV_EINVAL;
  if ((int64_t)a->sinks + a->recent > a->budget) return FP8KV_EINVAL;
  if (a->num_kv_heads > 65535 || a->max_len > (1 << 30)) return FP8KV_EUNSUPPORTED;
  if (a->batch == 0) return FP8KV_OK;
  if (!a->kv_len || !a->n_keep || !aligned(a->kv_len, 4) || !aligned(a->n_keep, 4) || !aligned(a->status, 4))
    return FP8KV_EINVAL;
  // a list reads its length while another one's first CTA writes the number kept
  if (overlap(a->kv_len, a->n_keep, a->batch)) return FP8KV_EINVAL;
  if (a->max_len > 0 && (!a->score || !a->keep)) return FP8KV_EINVAL;
  const int64_t s[] = {a->score_stride_req, a->score_stride_head, a->keep_stride_req, a->keep_stride_list};
  if (!aligned(a->score, 4) || !aligned(a->keep, 4) || !strides_ok(s, 4, 1)) return FP8KV_EINVAL;
  const int64_t most = a->budget < a->max_len ? a->budget : a->max_len;
  if (!apart(a->batch, s[2], a->lists, s[3], most)) return FP8KV_EINVAL;
  if ((int64_t)a->batch * a->lists > (1 << 27)) return FP8KV_EUNSUPPORTED;  // grid
  const int sms = sm_count();
  if (sms < 1) return FP8KV_ECUDA;
  return done(launch_cache_select(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int fp8kv_attn_cache_move(const fp8kv_cache_move_args* a, fp8kv_stream_t stream) {
  if (!a) return FP8KV_EINVAL;
  if (a->batch < 0 || a->num_kv_heads < 1 || a->max_count < 0 || a->page_size < 1 || a->max_blocks < 1 ||
      a->num_kv_blocks < 1)
    return FP8KV_EINVAL;
  if (a->lists != 1 && a->lists != a->num_kv_heads) return FP8KV_EINVAL;
  if (a->head_dim < 16 || a->head_dim > 1024 || a->head_dim % 16) return FP8KV_EINVAL;
  if (a->kv_format != FP8KV_KV_E4M3 && a->kv_format != FP8KV_KV_E5M2 && a->kv_format != FP8KV_KV_BF16)
    return FP8KV_EINVAL;
  if (a->num_kv_heads > 65535 || a->max_count > (1 << 30)) return FP8KV_EUNSUPPORTED;
  if (a->batch == 0 || a->max_count == 0) return FP8KV_OK;
  if (!a->k_cache || !a->v_cache || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16)) return FP8KV_EINVAL;
  const int64_t bs[] = {a->kc_stride_block, a->kc_stride_token, a->kc_stride_head,
                        a->vc_stride_block, a->vc_stride_token, a->vc_stride_head};
  if (!strides_ok(bs, 6, 16)) return FP8KV_EINVAL;
  if (!a->block_table || a->block_table_stride < a->max_blocks || !aligned(a->block_table, 4)) return FP8KV_EINVAL;
  if (a->dst_table == a->block_table) return FP8KV_EINVAL;  // (no order between reads and writes of the same pages)
  if (a->dst_table && (a->dst_max_blocks < 1 || a->dst_table_stride < a->dst_max_blocks || !aligned(a->dst_table, 4)))
    return FP8KV_EINVAL;
  if (!a->src || !a->count || !aligned(a->src, 4) || !aligned(a->count, 4) || !aligned(a->first, 4) ||
      !aligned(a->status, 4))
    return FP8KV_EINVAL;
  const int64_t es[] = {a->src_stride_req, a->src_stride_list, a->score_stride_req, a->score_stride_head,
                        a->score_out_stride_req, a->score_out_stride_head};
  if (!strides_ok(es, 6, 1)) return FP8KV_EINVAL;
  if (!a->score != !a->score_out) return FP8KV_EINVAL;
  if (a->score) {
    if (!aligned(a->score, 4) || !aligned(a->score_out, 4) || a->max_len < 1)
      return FP8KV_EINVAL;
    if (!apart(a->batch, es[4], a->num_kv_heads, es[5], a->max_len)) return FP8KV_EINVAL;
    // (weights are read while others are written, in no order)
    if (meet({a->batch, es[2], a->num_kv_heads, es[3]}, {a->batch, es[4], a->num_kv_heads, es[5]}, a->max_len,
             floats_between(a->score, a->score_out)))
      return FP8KV_EINVAL;
  }
  const int sms = sm_count();
  if (sms < 1) return FP8KV_ECUDA;
  return done(launch_cache_move(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
}
