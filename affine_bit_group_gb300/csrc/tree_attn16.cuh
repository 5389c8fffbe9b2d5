// Host launcher of the 16-bit tree_attn kernel (tree_attn16.cu).
#pragma once

#include "tree_attn.cuh"

namespace abg {

size_t tree_attn16_bytes(int D);
// early: the first launch may start before the launch ahead of it ends; pdl:
// the second before the first does; withhold: the ring item that no block
// brings (-1: none; abg_selftest_tree_attn_timeout)
cudaError_t launch_tree_attn16(const AttnArgs &p, void *ws, bool early, bool pdl, int withhold, cudaStream_t stream);

}  // namespace abg
