// kvq_attn over rows of 128 columns in 8 bits.
#include "abg_kernels.cuh"
#include "kvq_attn.cuh"

namespace abg {

template <>
cudaError_t kvq_attn_launch<128, 8>(const KvqAttnArgs &x, int group, int rt, bool split, void *ws, bool early, bool pdl,
                                  cudaStream_t stream) {
    return kvq_by_rows<128, 8>(group, rt, split, KvqGo{x, ws, early, pdl, stream});
}

}  // namespace abg
