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

// By the 16 lanes of a half warp (l: place in it; all 32 lanes call it): the rows
// u[r][0][0..V) at columns V*l.., u[r][1][..) at D/2 + V*l.. into codes and pairs, all
// rows' steps side by side.  rows[r]: the row's place in the cache (-1: not written)
// of keys, or (values[r]) of values.
template <int D, int R>
__device__ __forceinline__ void put_quantised(const float (&u)[R][2][D / 32], int l, const int64_t (&rows)[R],
                                              const bool (&values)[R], const abg_kvq_cache &c) {
    constexpr int V = D / 32, C = 2 * R;  // chunks of a lane, 2 r + h
    const int lane = threadIdx.x & 31, bits = c.bits, group = c.group;
    float lo[C], hi[C];
    const bool joined = group > D / 2;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float &a = lo[2 * r + h], &b = hi[2 * r + h];
            a = INFINITY, b = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                a = fminf(a, u[r][h][i]);
                b = fabsf(u[r][h][i]) <= kLargestHalf ? fmaxf(b, u[r][h][i]) : INFINITY;  // (a NaN too)
            }
        }
        if (joined) {
            lo[2 * r] = lo[2 * r + 1] = fminf(lo[2 * r], lo[2 * r + 1]);
            hi[2 * r] = hi[2 * r + 1] = fmaxf(hi[2 * r], hi[2 * r + 1]);
        }
    }
    // a group is at least C lanes' chunks: half of the chunks go to the other half of
    // the lanes in each step, until lane l has that of index l mod C
    const int lanes = min(16, group / V);
#pragma unroll
    for (int d = C / 2; d >= 1; d /= 2) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const float a = __shfl_xor_sync(0xffffffffu, up ? lo[i] : lo[i + d], d);
            const float b = __shfl_xor_sync(0xffffffffu, up ? hi[i] : hi[i + d], d);
            lo[i] = fminf(up ? lo[i + d] : lo[i], a);
            hi[i] = fmaxf(up ? hi[i + d] : hi[i], b);
        }
    }
    for (int d = C; d < lanes; d *= 2) {
        lo[0] = fminf(lo[0], __shfl_xor_sync(0xffffffffu, lo[0], d));
        hi[0] = fmaxf(hi[0], __shfl_xor_sync(0xffffffffu, hi[0], d));
    }
    const float levels = bits == 4 ? 15.0f : 255.0f;
    const bool bad = hi[0] == INFINITY;
    const __half nan = __ushort_as_half(0x7fff);
    const __half2 own = bad ? __halves2half2(nan, nan)
                            : __halves2half2(__float2half_rn(__fdiv_rn(__fsub_rn(hi[0], lo[0]), levels)), __float2half_rn(lo[0]));
    const float own_inv = __low2float(own) > 0.0f ? __frcp_rn(__low2float(own)) : 0.0f;  // (a NaN: 0)
    const uint32_t own_pair = *reinterpret_cast<const uint32_t *>(&own);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        unsigned char *codes = static_cast<unsigned char *>(values[r] ? c.Vc : c.Kc) + rows[r] * (D * bits / 8);
        uint32_t *pairs = static_cast<uint32_t *>(values[r] ? c.Vs : c.Ks) + rows[r] * (D / group);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int from = (lane & ~(C - 1)) + 2 * r + h;
            const uint32_t pair = __shfl_sync(0xffffffffu, own_pair, from);
            const float inv = __shfl_sync(0xffffffffu, own_inv, from);
            const float b = __half2float(__ushort_as_half(static_cast<unsigned short>(pair >> 16)));
            uint32_t code[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // clamped, then rounded to a whole number by 1.5 * 2^23 (a NaN: 0, as 0 * NaN is clamped to 0)
                const float x = fminf(fmaxf(__fmul_rn(__fsub_rn(u[r][h][i], b), inv), 0.0f), levels);
                code[i] = __float_as_uint(__fadd_rn(x, 12582912.0f)) & 255u;
            }
            const int col = h * (D / 2) + V * l;
            if (rows[r] >= 0) {
                store_codes<V>(codes + col * bits / 8, code, bits);
                if (l % lanes == 0 && !(joined && h)) pairs[col / group] = pair;
            }
        }
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
    // (no launch after this one starts early: some read caches and weights before they wait)
    grid_dep_wait();
    struct Token {
        int64_t n, src, slot;
        int32_t pos;
        int h0;
    };
    // all tokens' last heads (keys and values, the longest work) first, so that every
    // warp has its share of each kind
    auto token = [&](int64_t unit) {
        Token t{0, -1, -1, 0, 0};
        if (unit >= units) return t;
        const int64_t g = div_up_to_64(unit, a.N);
        t.n = unit - g * a.N;
        t.h0 = (groups - 1 - static_cast<int>(g)) * P::kHeads;
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
            int64_t rows[kSteps];
            bool values[kSteps];
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
                if (h < nq) {
                    T *to = static_cast<T *>(a.qo) + (t.n * a.Hq + h) * D;
                    store_e<T, V>(to + V * l, u[r][0]);
                    store_e<T, V>(to + D / 2 + V * l, u[r][1]);
                }
                values[r] = h >= nq + nk;
                rows[r] = kept && h >= nq && h < heads ? base + (values[r] ? h - nq - nk : h - nq) * a.c.page : -1;
            }
            if (t.h0 + P::kHeads > nq) put_quantised<D>(u, l, rows, values, a.c);  // (the whole warp, or none of it)
        }
        t = next;
    }
}

// ------------------------------------------------------------- kvq_get -----
// A block a tile of tokens, whose rows it finds once; then a thread eight columns at
// a time, one or two words and a pair in, 16 or 32 bytes out, the columns first, then
// heads, K and V, tokens, so that a warp reads and writes whole rows.  Four such
// places at a time a thread, so that their words are on their way together.
constexpr int kGetThreads = 256, kGetEach = 4, kGetTokens = 128;

// Byte k of w as a float (0x4b000000 + c is 2^23 + c).
template <int k>
__device__ __forceinline__ float byte_value(uint32_t w) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + k)) - 8388608.0f;
}

template <typename T, int kBits>
__global__ void __launch_bounds__(kGetThreads) kvq_get_kernel(const __grid_constant__ abg_kvq_get_args a, int kinds,
                                                              int log_cols, int tokens) {
    __shared__ int64_t s_row[kGetTokens];  // of head 0; -1: none
    const int tid = threadIdx.x, Hkv = static_cast<int>(a.c.Hkv);
    const int per = kinds * Hkv << log_cols, log_pair = a.c.group == 32 ? 2 : 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * tokens;
    const int here = static_cast<int>(min(static_cast<int64_t>(tokens), a.N - n0)), items = here * per;
    grid_dep_wait();  // (and nothing after this one starts early, as kvq_put)
    if (tid < here) {
        const int64_t slot = a.slots ? a.slots[n0 + tid] : n0 + tid;
        int64_t row = -1;
        if (slot >= 0 && slot < a.c.pages * a.c.page) {
            const int64_t page = div_up_to_64(slot, a.c.page);
            row = page * Hkv * a.c.page + (slot - page * a.c.page);
        }
        s_row[tid] = row;
    }
    __syncthreads();
    for (int i0 = tid; i0 < items; i0 += kGetEach * kGetThreads) {
        int n[kGetEach], h[kGetEach], col[kGetEach];
        bool value[kGetEach];
        uint2 w[kGetEach];
        float2 f[kGetEach];
#pragma unroll
        for (int k = 0; k < kGetEach; ++k) {
            const int i = i0 + k * kGetThreads;
            n[k] = -1;
            w[k] = make_uint2(0, 0);
            f[k] = make_float2(0.0f, 0.0f);
            if (i >= items) continue;
            n[k] = static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(per));
            const int rest = i - n[k] * per, kh = rest >> log_cols;
            col[k] = rest & ((1 << log_cols) - 1);
            value[k] = kh >= Hkv || !a.k;
            h[k] = kh >= Hkv ? kh - Hkv : kh;
            const int64_t row = s_row[n[k]];
            if (row < 0) continue;
            const int64_t at = ((row + h[k] * a.c.page) << log_cols) + col[k];
            const void *codes = value[k] ? a.c.Vc : a.c.Kc;
            if constexpr (kBits == 4) {
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
            if constexpr (kBits == 4) {
                const uint32_t even = w[k].x & 0x0f0f0f0fu, odd = w[k].x >> 4 & 0x0f0f0f0fu;
                v[0] = byte_value<0>(even), v[1] = byte_value<0>(odd), v[2] = byte_value<1>(even), v[3] = byte_value<1>(odd);
                v[4] = byte_value<2>(even), v[5] = byte_value<2>(odd), v[6] = byte_value<3>(even), v[7] = byte_value<3>(odd);
            } else {
                v[0] = byte_value<0>(w[k].x), v[1] = byte_value<1>(w[k].x), v[2] = byte_value<2>(w[k].x);
                v[3] = byte_value<3>(w[k].x), v[4] = byte_value<0>(w[k].y), v[5] = byte_value<1>(w[k].y);
                v[6] = byte_value<2>(w[k].y), v[7] = byte_value<3>(w[k].y);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(f[k].x, v[i], f[k].y);  // (the product is exact: 11 and 8 bits)
            T *to = static_cast<T *>(value[k] ? a.v : a.k) + (n0 + n[k]) * (value[k] ? a.v_row : a.k_row) +
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

template <typename T, int kBits>
cudaError_t get_bits(const abg_kvq_get_args &a, bool pdl, cudaStream_t stream) {
    const int kinds = (a.k != nullptr) + (a.v != nullptr);
    const int log_cols = a.c.D == 64 ? 3 : a.c.D == 128 ? 4 : 5;
    const int64_t per = kinds * a.c.Hkv << log_cols;
    // eight places a thread, as long as there are four blocks an SM
    const int64_t tokens = std::max<int64_t>(
        1, std::min<int64_t>({kGetTokens, 2 * kGetEach * kGetThreads / per, a.N / (4ll * sm_count())}));
    return launch_kernel(kvq_get_kernel<T, kBits>, dim3(static_cast<unsigned>((a.N + tokens - 1) / tokens)),
                         dim3(kGetThreads), 0, stream, pdl && !capturing(stream), a, kinds, log_cols,
                         static_cast<int>(tokens));
}
template <typename T>
cudaError_t get(const abg_kvq_get_args &a, bool pdl, cudaStream_t stream) {
    return a.c.bits == 4 ? get_bits<T, 4>(a, pdl, stream) : get_bits<T, 8>(a, pdl, stream);
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
