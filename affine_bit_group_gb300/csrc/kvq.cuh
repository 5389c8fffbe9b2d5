// Host launchers of the quantised cache's kernels (kvq.cu, kvq_attn.cu).
#pragma once

#include "../../include/abg.h"

#include <cuda_runtime.h>

namespace abg {

cudaError_t launch_kvq_put(const abg_kvq_put_args &a, bool pdl, cudaStream_t stream);
cudaError_t launch_kvq_get(const abg_kvq_get_args &a, bool pdl, cudaStream_t stream);

size_t kvq_attn_bytes(const abg_kvq_cache &c, int64_t Hq, int64_t max_span, int type);
cudaError_t launch_kvq_attn(const abg_kvq_attn_args &a, void *ws, bool pdl, cudaStream_t stream);

}  // namespace abg
