// Host launchers of the draft-verification kernels (draft.cu, tree_attn.cu).
#pragma once

#include "../../include/abg.h"

#include <cuda_runtime.h>

namespace abg {

// Launches a kernel; with `pdl` it may start before the launch ahead of it on
// the stream has finished (it then waits with grid_dep_wait).
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*fn)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                          A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

// Whether the stream is being captured: then a call's first launch does not
// start early, since the node ahead of it need not be a kernel.
inline bool capturing(cudaStream_t stream) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    return cudaStreamIsCapturing(stream, &st) != cudaSuccess || st != cudaStreamCaptureStatusNone;
}

// The request that owns row n: the last b with cu[b] <= n, in 0 .. B-1.
__device__ __forceinline__ int request_of(const int32_t *cu, int B, int n) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= n) {
            lo = mid;
        } else {
            hi = mid - 1;
        }
    }
    return lo;
}

struct PagePlanArgs {
    const int32_t *lens, *add, *cu, *held;
    const int64_t *ends;
    int32_t *ring, *table;
    int64_t *slots;
    int32_t *pos, *lens_out, *held_out;
    int64_t *ends_out;
    int32_t *info;
    int B, N, page, width, ring_len;
};
// pdl: the launches may start before the launch ahead of them has finished
// (they wait for it before they read anything)
cudaError_t launch_page_plan(const PagePlanArgs &a, bool pdl, cudaStream_t stream);

cudaError_t launch_tree_plan(const int32_t *parent, const int32_t *lens, const int32_t *cu, uint64_t *mask,
                             int32_t *pos, int B, int N, int words, bool pdl, cudaStream_t stream);

cudaError_t launch_kv_put(const abg_kv_put_args &a, bool pdl, cudaStream_t stream);

size_t tree_accept_bytes(int64_t N, int64_t V);
cudaError_t launch_tree_accept(const float *logits, int64_t ld, const int32_t *tok, const int32_t *parent,
                               const int32_t *cu, int32_t *best, int32_t *rows, int32_t *add, int32_t *last, int B,
                               int N, int64_t V, void *ws, bool pdl, cudaStream_t stream);

size_t tree_attn_bytes(int Hq, int Hkv, int D, int max_span, int type);
// withhold: as launch_tree_attn16's
cudaError_t launch_tree_attn(const abg_tree_attn_args &a, void *ws, bool pdl, int withhold, cudaStream_t stream);

// the 16-bit kernel's device status word (OR-ed into *bits)
cudaError_t tree_attn16_status(unsigned *bits, bool clear);

// Whether launches may start early (the environment's ABG_PDL; api.cu).
bool early_launches();

// Records e as the calling thread's last CUDA error (api.cu) and returns the
// call's status.
abg_status cuda_status(cudaError_t e, const char *where);

}  // namespace abg
