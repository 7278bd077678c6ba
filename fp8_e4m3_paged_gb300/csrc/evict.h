// Declarations shared by the units that score, select and move cached positions.
#pragma once

#include <cuda_runtime.h>

#include "fp8kv_attn.h"

namespace fp8kv {

cudaError_t launch_cache_select(const fp8kv_cache_select_args& a, int sms, cudaStream_t s);
cudaError_t launch_cache_move(const fp8kv_cache_move_args& a, int sms, cudaStream_t s);

}  // namespace fp8kv
