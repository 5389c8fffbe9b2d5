// Rows of keys, values and queries: loads and stores of a thread's columns in
// the three types, and the division that finds a token's page.
#pragma once

#include "abg_dev.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

namespace abg {

template <typename T>
__device__ __forceinline__ float widen(T v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else {
        return static_cast<float>(v);
    }
}
template <typename T>
__device__ __forceinline__ T narrow(float v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        return __float2bfloat16_rn(v);
    } else {
        return __float2half_rn(v);
    }
}

// a / b of nonnegative numbers, in 32 bits where they fit (64-bit division is
// a long subroutine)
__device__ __forceinline__ int64_t div_up_to_64(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// E consecutive values, E * sizeof(T) = 4, 8, 16 or 32 bytes
template <typename T, int E>
__device__ __forceinline__ void load_e(const T *p, float (&v)[E]) {
    constexpr int kBytes = E * sizeof(T);
    alignas(16) T t[E];
    if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t *>(t) = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2 *>(t) = *reinterpret_cast<const uint2 *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            reinterpret_cast<uint4 *>(t)[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = widen(t[i]);
}
template <typename T, int E>
__device__ __forceinline__ void store_e(T *p, const float (&v)[E]) {
    constexpr int kBytes = E * sizeof(T);
    alignas(16) T t[E];
#pragma unroll
    for (int i = 0; i < E; ++i) t[i] = narrow<T>(v[i]);
    if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<uint32_t *>(t);
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(t);
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<uint4 *>(t)[i];
    }
}

}  // namespace abg
