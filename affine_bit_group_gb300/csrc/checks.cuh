// What the C entries of the cache's calls check of their arguments.
#pragma once

#include "../../include/abg.h"

#include <cuda_runtime.h>

#include <initializer_list>

namespace abg {

constexpr int64_t kMax32 = 0x7fffffff;

inline bool on(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

struct Span {
    uintptr_t lo, hi;
};
inline Span span(const void *p, int64_t count, size_t elem) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, p ? lo + static_cast<uintptr_t>(count) * elem : lo};
}
// No output may overlap an input or another output.
inline bool apart(std::initializer_list<Span> out, std::initializer_list<Span> in) {
    auto meet = [](Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; };
    for (auto o = out.begin(); o != out.end(); ++o) {
        for (auto p = out.begin(); p != o; ++p)
            if (meet(*o, *p)) return false;
        for (const Span &i : in)
            if (meet(*o, i)) return false;
    }
    return true;
}

inline bool known_type(int t) { return t >= ABG_SB_F32 && t <= ABG_SB_F16; }
inline int64_t elem(int t) { return t == ABG_SB_F32 ? 4 : 2; }
inline bool known_width(int64_t D) { return D == 64 || D == 128 || D == 256; }
// a product of positive factors that stays below 2^62
inline bool bounded(std::initializer_list<int64_t> f) {
    int64_t n = 1;
    for (int64_t v : f) {
        if (v < 0) return false;
        if (v > 0 && n > (int64_t(1) << 62) / v) return false;
        n *= v > 0 ? v : 1;
    }
    return true;
}
inline cudaStream_t to_stream(void *s) { return static_cast<cudaStream_t>(s); }

}  // namespace abg
