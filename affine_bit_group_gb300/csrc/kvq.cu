// Rows into and out of the quantised cache: kvq_put and kvq_get (formulas in
// include/abg.h).
//
// The norm and rotation are the steps of the single-token attention ("Metal:
// queued rmsq, swq, gdn and atq kernels ...", bendlang/bend #1440, Change, the
// Array.atq bullet), and the format is that of the weights; the rest has no
// counterpart on the pages.
#include "abg_kernels.cuh"
#include "draft.cuh"
#include "kv_rows.cuh"
#include "kvq.cuh"

#include <algorithm>

namespace abg {

namespace {

constexpr float kLargestHalf = 65504.0f;

// ------------------------------------------------------------- kvq_put -----
// kv_put's lanes and steps up to the rotated row: a warp a token and 8 of its
// heads (4 of 256 columns), two at a time, lane l of a half warp with columns
// V*l .. V*l+V-1 of a head (V = D/32) and the ones D/2 further on.  A group is then
// in 4, 8 or 16 lanes' chunks of one half of the columns, or (64 columns a row, one
// group) in all 16 lanes' both chunks, and its least and largest value meet by
// shuffles; the lanes then quantise and pack their own columns.
constexpr int kPutWarps = 8;

// V codes of `bits` bits, low first, to p (V*bits/8 bytes, aligned to as many).
template <int V>
__device__ __forceinline__ void store_codes(unsigned char *p, const uint32_t (&code)[V], int bits) {
    if (bits == 4) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) w |= code[i] << (4 * i);
        if constexpr (V == 2) {
            *p = static_cast<unsigned char>(w);
        } else if constexpr (V == 4) {
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w);
        } else {
            *reinterpret_cast<uint32_t *>(p) = w;
        }
    } else {
        uint32_t w[(V + 3) / 4] = {};
#pragma unroll
        for (int i = 0; i < V; ++i) w[i / 4] |= code[i] << (8 * (i % 4));
        if constexpr (V == 2) {
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
        } else if constexpr (V == 4) {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        } else {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        }
    }
}

// By the 16 lanes of a half warp (l: place in it; all 32 lanes call it): the row
// u[0][0..V) at columns V*l.., u[1][..) at D/2 + V*l.. into codes and pairs; `kept`:
// whether the row is to be written.
template <int D>
__device__ __forceinline__ void put_quantised(const float (&u)[2][D / 32], int l, bool kept, int bits, int group,
                                              unsigned char *codes, __half2 *pairs) {
    constexpr int V = D / 32;
    float lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        lo[h] = INFINITY;
        hi[h] = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            lo[h] = fminf(lo[h], u[h][i]);
            hi[h] = fabsf(u[h][i]) <= kLargestHalf ? fmaxf(hi[h], u[h][i]) : INFINITY;  // (a NaN too)
        }
    }
    const bool joined = group > D / 2;
    if (joined) lo[0] = lo[1] = fminf(lo[0], lo[1]), hi[0] = hi[1] = fmaxf(hi[0], hi[1]);
    const int lanes = min(16, group / V);  // of a group's chunks of one half
    for (int d = 1; d < lanes; d <<= 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            lo[h] = fminf(lo[h], __shfl_xor_sync(0xffffffffu, lo[h], d));
            hi[h] = fmaxf(hi[h], __shfl_xor_sync(0xffffffffu, hi[h], d));
        }
    }
    if (!kept) return;
    const float levels = bits == 4 ? 15.0f : 255.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool bad = hi[h] == INFINITY;
        const __half bias = bad ? __ushort_as_half(0x7fff) : __float2half_rn(lo[h]);
        const __half scale =
            bad ? __ushort_as_half(0x7fff) : __float2half_rn(__fdiv_rn(__fsub_rn(hi[h], lo[h]), levels));
        const float b = __half2float(bias), s = __half2float(scale);
        const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;  // (a NaN: 0)
        uint32_t code[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = rintf(__fmul_rn(__fsub_rn(u[h][i], b), inv));
            code[i] = bad ? 0u : static_cast<uint32_t>(fminf(fmaxf(x, 0.0f), levels));
        }
        const int col = h * (D / 2) + V * l;
        store_codes<V>(codes + col * bits / 8, code, bits);
        if (l % lanes == 0 && !(joined && h)) pairs[col / group] = __halves2half2(scale, bias);
    }
}

template <typename S, typename T, int D>
__global__ void __launch_bounds__(32 * kPutWarps, D == 256 ? 2 : 3) kvq_put_kernel(
    const __grid_constant__ abg_kvq_put_args a, int groups) {
    using P = Put<D>;
    constexpr int V = P::V, kSteps = P::kSteps;
    const int lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
    const int64_t units = a.N * groups, stride = static_cast<int64_t>(gridDim.x) * kPutWarps;
    const int nq = a.q ? static_cast<int>(a.Hq) : 0, nk = static_cast<int>(a.c.Hkv), heads = nq + 2 * nk;
    const int row_bytes = D * a.c.bits / 8, row_pairs = D / a.c.group;
    // (no launch after this one starts early: some read caches and weights before they wait)
    grid_dep_wait();
    struct Token {
        int64_t n, src, slot;
        int32_t pos;
        int h0;
    };
    auto token = [&](int64_t unit) {
        Token t{0, -1, -1, 0, 0};
        if (unit >= units) return t;
        t.n = div_up_to_64(unit, groups);
        t.h0 = static_cast<int>(unit - t.n * groups) * P::kHeads;
        t.src = a.rows ? a.rows[t.n] : t.n;
        t.slot = a.slots ? a.slots[t.n] : t.n;
        if (a.cos) t.pos = a.pos[t.n];
        return t;
    };
    int64_t unit = static_cast<int64_t>(blockIdx.x) * kPutWarps + (threadIdx.x >> 5);
    Token t = token(unit);
    for (; unit < units; unit += stride) {
        const Token next = token(unit + stride);
        if (t.src >= 0 && t.src < a.src_rows) {
            float u[kSteps][2][V], c[V], s[V];
#pragma unroll
            for (int r = 0; r < kSteps; ++r) {
                const int h = t.h0 + 2 * r + half;
                if (h >= heads) continue;
                const S *p = h < nq        ? static_cast<const S *>(a.q) + t.src * a.q_row + h * a.q_head
                             : h < nq + nk ? static_cast<const S *>(a.k) + t.src * a.k_row + (h - nq) * a.k_head
                                           : static_cast<const S *>(a.v) + t.src * a.v_row + (h - nq - nk) * a.v_head;
                load_e<S, V>(p + V * l, u[r][0]);
                load_e<S, V>(p + D / 2 + V * l, u[r][1]);
            }
            if (a.cos && t.h0 < nq + nk) {
                const bool in = t.pos >= 0 && t.pos < a.cos_rows;
                const int64_t at = (in ? t.pos : 0) * static_cast<int64_t>(D / 2) + V * l;
                load_e<float, V>(a.cos + at, c);
                load_e<float, V>(a.sin + at, s);
                if (!in)
#pragma unroll
                    for (int i = 0; i < V; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
            }
            float factor = 0.0f;  // lane r of a half: of the half's head of step r
            if ((a.qn_w && t.h0 < nq) || (a.kn_w && t.h0 < nq + nk && t.h0 + P::kHeads > nq)) {
                float ss = 0.0f;
#pragma unroll
                for (int r = 0; r < kSteps; ++r) {
                    const float lo = chunk_tree<V>(u[r][0]), hi = chunk_tree<V>(u[r][1]);
                    // even lanes go on with the lower columns' sum, odd ones with the upper's
                    const float away = __shfl_xor_sync(0xffffffffu, l & 1 ? lo : hi, 1);
                    float sum = __fadd_rn(l & 1 ? hi : lo, away);
#pragma unroll
                    for (int d = 2; d < 16; d <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
                    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 1));
                    if (l == r) ss = sum;
                }
                factor = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(D)), a.eps)));
            }
            const bool kept = t.slot >= 0 && t.slot < a.c.pages * a.c.page;
            const int64_t page = kept ? div_up_to_64(t.slot, a.c.page) : 0;
            const int64_t base = page * a.c.Hkv * a.c.page + (t.slot - page * a.c.page);
#pragma unroll
            for (int r = 0; r < kSteps; ++r) {
                const int h = t.h0 + 2 * r + half;
                const float f = __shfl_sync(0xffffffffu, factor, r, 16);
                if (h < nq + nk) {
                    const float *w = h < nq ? a.qn_w : a.kn_w;
                    if (w) {
                        float wv[2][V];
                        load_e<float, V>(w + V * l, wv[0]);
                        load_e<float, V>(w + D / 2 + V * l, wv[1]);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            u[r][0][i] = __fmul_rn(__fmul_rn(u[r][0][i], f), wv[0][i]);
                            u[r][1][i] = __fmul_rn(__fmul_rn(u[r][1][i], f), wv[1][i]);
                        }
                    }
                    if (a.cos) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float x = u[r][0][i], y = u[r][1][i];
                            u[r][0][i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
                            u[r][1][i] = __fadd_rn(__fmul_rn(y, c[i]), __fmul_rn(x, s[i]));
                        }
                    }
                }
                const bool value = h >= nq + nk;
                if (h < nq) {
                    T *to = static_cast<T *>(a.qo) + (t.n * a.Hq + h) * D;
                    store_e<T, V>(to + V * l, u[r][0]);
                    store_e<T, V>(to + D / 2 + V * l, u[r][1]);
                }
                if (t.h0 + 2 * r + 1 < nq || t.h0 + 2 * r >= heads) continue;  // (the whole warp: no row of the cache)
                const int64_t row = base + (value ? h - nq - nk : h - nq) * a.c.page;
                put_quantised<D>(u[r], l, kept && h >= nq && h < heads, a.c.bits, a.c.group,
                                 static_cast<unsigned char *>(value ? a.c.Vc : a.c.Kc) + row * row_bytes,
                                 static_cast<__half2 *>(value ? a.c.Vs : a.c.Ks) + row * row_pairs);
            }
        }
        t = next;
    }
}

// ------------------------------------------------------------- kvq_get -----
// A thread eight columns: one or two words and a pair in, 16 or 32 bytes out.
// Threads go over (row, key or value, head, eight columns), the columns first, so
// that a warp reads and writes whole rows; four such places at a time a thread, so
// that their slots, then their words, are on their way together.
constexpr int kGetThreads = 256, kGetEach = 4;

template <typename T>
__global__ void __launch_bounds__(kGetThreads) kvq_get_kernel(const __grid_constant__ abg_kvq_get_args a, int kinds,
                                                              int log_cols) {
    grid_dep_wait();  // (and nothing after this one starts early, as kvq_put)
    const int cols = 1 << log_cols, log_pair = a.c.group == 32 ? 2 : 3;        // eights of a row and of a pair
    const int64_t Hkv = a.c.Hkv, per = kinds * Hkv, all = a.N * per << log_cols;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kGetThreads, slots = a.c.pages * a.c.page;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kGetThreads + threadIdx.x; i0 < all; i0 += kGetEach * stride) {
        int64_t n[kGetEach], slot[kGetEach];
        int h[kGetEach], col[kGetEach];
        bool value[kGetEach];
#pragma unroll
        for (int k = 0; k < kGetEach; ++k) {
            const int64_t i = i0 + k * stride;
            n[k] = -1;
            if (i >= all) continue;
            col[k] = static_cast<int>(i & (cols - 1));
            n[k] = div_up_to_64(i >> log_cols, per);
            const int kh = static_cast<int>((i >> log_cols) - n[k] * per);
            value[k] = kh >= Hkv || !a.k;
            h[k] = kh >= Hkv ? kh - static_cast<int>(Hkv) : kh;
            slot[k] = a.slots ? a.slots[n[k]] : n[k];
        }
        uint2 w[kGetEach];
        float2 f[kGetEach];
#pragma unroll
        for (int k = 0; k < kGetEach; ++k) {
            w[k] = make_uint2(0, 0);
            f[k] = make_float2(0.0f, 0.0f);
            if (n[k] < 0 || slot[k] < 0 || slot[k] >= slots) continue;
            const int64_t page = div_up_to_64(slot[k], a.c.page);
            const int64_t row = (page * Hkv + h[k]) * a.c.page + (slot[k] - page * a.c.page);
            const int64_t at = (row << log_cols) + col[k];
            const void *codes = value[k] ? a.c.Vc : a.c.Kc;
            if (a.c.bits == 4) {
                w[k].x = static_cast<const uint32_t *>(codes)[at];
            } else {
                w[k] = static_cast<const uint2 *>(codes)[at];
            }
            f[k] = __half22float2(static_cast<const __half2 *>(value[k] ? a.c.Vs : a.c.Ks)[at >> log_pair]);
        }
#pragma unroll
        for (int k = 0; k < kGetEach; ++k) {
            if (n[k] < 0) continue;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t code =
                    a.c.bits == 4 ? w[k].x >> (4 * i) & 15u : (i < 4 ? w[k].x : w[k].y) >> (8 * (i % 4)) & 255u;
                // (the product is exact: 11 and 8 bits)
                v[i] = __fadd_rn(__fmul_rn(f[k].x, static_cast<float>(code)), f[k].y);
            }
            T *to = static_cast<T *>(value[k] ? a.v : a.k) + n[k] * (value[k] ? a.v_row : a.k_row) +
                    h[k] * (value[k] ? a.v_head : a.k_head) + 8 * col[k];
            store_e<T, 8>(to, v);
        }
    }
}

template <typename S, typename T, int D>
cudaError_t put_d(const abg_kvq_put_args &a, bool early, cudaStream_t stream) {
    // as many blocks as fit at once
    static const int fit = [] {
        int per = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kvq_put_kernel<S, T, D>, 32 * kPutWarps, 0) !=
            cudaSuccess)
            per = 1;
        return std::max(per, 1) * sm_count();
    }();
    const int heads = static_cast<int>((a.q ? a.Hq : 0) + 2 * a.c.Hkv);
    const int groups = (heads + Put<D>::kHeads - 1) / Put<D>::kHeads;
    const int64_t blocks = (a.N * groups + kPutWarps - 1) / kPutWarps;
    return launch_kernel(kvq_put_kernel<S, T, D>, dim3(static_cast<unsigned>(std::min<int64_t>(blocks, fit))),
                         dim3(32 * kPutWarps), 0, stream, early, a, groups);
}
template <typename S, typename T>
cudaError_t put(const abg_kvq_put_args &a, bool early, cudaStream_t stream) {
    return a.c.D == 64    ? put_d<S, T, 64>(a, early, stream)
           : a.c.D == 128 ? put_d<S, T, 128>(a, early, stream)
                          : put_d<S, T, 256>(a, early, stream);
}

template <typename T>
cudaError_t get(const abg_kvq_get_args &a, bool pdl, cudaStream_t stream) {
    const int kinds = (a.k != nullptr) + (a.v != nullptr);
    const int log_cols = a.c.D == 64 ? 3 : a.c.D == 128 ? 4 : 5;
    const int64_t threads = a.N * kinds * a.c.Hkv << log_cols, each = kGetThreads * kGetEach;
    const int64_t blocks = std::min<int64_t>((threads + each - 1) / each, 8ll * sm_count());
    return launch_kernel(kvq_get_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kGetThreads), 0, stream,
                         pdl && !capturing(stream), a, kinds, log_cols);
}

}  // namespace

cudaError_t launch_kvq_put(const abg_kvq_put_args &a, bool pdl, cudaStream_t stream) {
    const bool early = pdl && !capturing(stream);
    switch (a.src_type) {
    case ABG_SB_F32:
        return !a.q || a.q_type == ABG_SB_F32  ? put<float, float>(a, early, stream)
               : a.q_type == ABG_SB_BF16       ? put<float, __nv_bfloat16>(a, early, stream)
                                               : put<float, __half>(a, early, stream);
    case ABG_SB_BF16: return put<__nv_bfloat16, __nv_bfloat16>(a, early, stream);
    default: return put<__half, __half>(a, early, stream);
    }
}

cudaError_t launch_kvq_get(const abg_kvq_get_args &a, bool pdl, cudaStream_t stream) {
    switch (a.type) {
    case ABG_SB_F32: return get<float>(a, pdl, stream);
    case ABG_SB_BF16: return get<__nv_bfloat16>(a, pdl, stream);
    default: return get<__half>(a, pdl, stream);
    }
}

}  // namespace abg
