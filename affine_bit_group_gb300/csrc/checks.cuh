// What the C entries of the cache's calls check of their arguments.
#pragma once

#include "../../include/abg.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <initializer_list>
#include <utility>

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

// [N] rows of H heads of D columns, at these strides (that of a single row or head
// does not count).
struct RowStrides {
    int64_t row, head;
};
// Rows that do not lie in one another: the heads of a row side by side before the
// next row, or the rows of a head before the next.
inline bool rows_apart(RowStrides s, int64_t N, int64_t H, int64_t D) {
    return (N == 1 && H == 1) || ((H == 1 || s.head >= D) && (N == 1 || s.row >= (H - 1) * s.head + D)) ||
           ((N == 1 || s.row >= D) && (H == 1 || s.head >= (N - 1) * s.row + D));
}
// Whether two such sets of rows (each rows_apart), the second `off` >= 0 columns on, have
// no column in common.  Exact at the same strides: the distances between their rows are
// off + i*row + j*head, |i| < N, |j| < H, and none is below D.  At other ones only where
// each row of the one (all its heads) lies between two of the other's, or each head (all
// its rows) between two heads.
inline bool rows_between(int64_t off, RowStrides a, RowStrides b, int64_t N, int64_t H, int64_t D) {
    if ((N == 1 || a.row == b.row) && (H == 1 || a.head == b.head)) {
        // the shorter of the two axes step by step, the next multiples of the other one's stride
        int64_t n = N, step = N == 1 ? 0 : a.row, h = H, each = H == 1 ? 0 : a.head;
        if (n < h) std::swap(n, h), std::swap(step, each);
        for (int64_t j = 1 - h; j < h; ++j) {
            const int64_t x = off + j * each;  // x - i*step, 1 - n <= i < n
            const int64_t low = n == 1 ? 0 : std::clamp(x / step - (x % step < 0), 1 - n, n - 2);
            for (int64_t i = low; i <= low + (n > 1); ++i)
                if (std::abs(x - i * step) < D) return false;
        }
        return true;
    }
    auto within = [off](int64_t a_period, int64_t b_period, int64_t a_extent, int64_t b_extent) {
        return a_period > 0 && a_period == b_period && off % a_period >= a_extent && off % a_period + b_extent <= a_period;
    };
    return within(a.row, b.row, (H - 1) * a.head + D, (H - 1) * b.head + D) ||
           within(a.head, b.head, (N - 1) * a.row + D, (N - 1) * b.row + D);
}
inline cudaStream_t to_stream(void *s) { return static_cast<cudaStream_t>(s); }

}  // namespace abg
