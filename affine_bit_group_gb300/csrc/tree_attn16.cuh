// Host launcher of the 16-bit tree_attn kernel (tree_attn16.cu).
#pragma once

#include "tree_attn.cuh"

namespace abg {

size_t tree_attn16_bytes(int D);
// early: the first launch may start before the launch ahead of it ends; pdl:
// the second before the first does
cudaError_t launch_tree_attn16(const AttnArgs &p, void *ws, bool early, bool pdl, cudaStream_t stream);

}  // namespace abg
