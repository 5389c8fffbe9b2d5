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
// kv_put's lanes and steps up to the rotated row: a warp a token and 4 of its
// heads, two at a time, lane l of a half warp with columns
// V*l .. V*l+V-1 of a head (V = D/32) and the ones D/2 further on.  A group is then
// in 4, 8 or 16 lanes' chunks of one half of the columns, or (64 columns a row, one
// group) in all 16 lanes' both chunks, and its least and largest value meet by
// shuffles; the lanes then quantise and pack their own columns.  A warp's next rows and
// rotations come to shared memory by cp.async meanwhile, each lane's own.  Instructions
// and their latency bound it alike: 8191 tokens of 16 + 4 + 4 heads of 128 columns, f32 to 4
// bits, with q in bf16, in 30.9 us (143 MB, 4.6 TB/s; kv_put to bf16 33) and 25.9 M warp
// instructions; with 8 heads a warp, for which two blocks an SM have registers, 20.3 M in
// 31.2, with four blocks, which spill, 33.5.  (Of f32 rows of 256 columns the ring has room
// for two of the three blocks: 8 + 2 + 2 heads 46.0 us, 45.1 compiled for two, q in f32 53.0
// either way; of bf16 rows 26.5 for three, 26.8 for two.)
// Loaded only when their turn came the rows took 38, with heads' places and 64-bit
// divisions for each token 34.6.  Calls so short that no warp has a second unit take two
// heads a warp and load them to registers: 8 tokens of 8 + 2 + 2 heads of 256 columns 3.0 us
// for 3.4, with the ring 4.1.
constexpr int kPutWarps = 8;

// kOnce: no warp has a second unit.
template <int D, bool kOnce>
struct PutUnit {
    static constexpr int V = D / 32;                // columns of a chunk
    static constexpr int kSteps = kOnce ? 1 : 2;    // heads of a half warp
    static constexpr int kHeads = 2 * kSteps;
    static constexpr int kBlocks = kOnce ? 4 : 3;   // an SM
};

// Least and largest; a NaN stays.
__device__ __forceinline__ float least(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float largest(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Pairwise tree of V squares, as kv_put's, the products in pairs.
template <int V>
__device__ __forceinline__ float square_tree(const float (&u)[V]) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const float2 y = mul2(make_float2(u[i], u[i + 1]), make_float2(u[i], u[i + 1]));
        x[i] = y.x, x[i + 1] = y.y;
    }
#pragma unroll
    for (int k = V / 2; k >= 1; k >>= 1)
#pragma unroll
        for (int i = 0; i < k; ++i) x[i] = __fadd_rn(x[2 * i], x[2 * i + 1]);
    return x[0];
}

// N codes of kBits bits, low first, in a word, of whole numbers x + 1.5 * 2^23: their bits
// are 0x4b400000 + x.
template <int kBits, int N>
__device__ __forceinline__ uint32_t code_word(const float *x) {
    uint32_t w = 0, over = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w += __float_as_uint(x[i]) << (kBits * i);
        over += 0x4b400000u << (kBits * i);
    }
    return w - over;
}
// V codes to p (V*kBits/8 bytes, aligned to as many).
template <int kBits, int V>
__device__ __forceinline__ void store_codes(unsigned char *p, const float (&x)[V]) {
    constexpr int kBytes = V * kBits / 8;
    if constexpr (kBytes == 1) {
        *p = static_cast<unsigned char>(code_word<kBits, V>(x));
    } else if constexpr (kBytes == 2) {
        *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(code_word<kBits, V>(x));
    } else if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t *>(p) = code_word<kBits, V>(x);
    } else {
        *reinterpret_cast<uint2 *>(p) = make_uint2(code_word<kBits, V / 2>(x), code_word<kBits, V / 2>(x + V / 2));
    }
}

// By the 16 lanes of a half warp (l: place in it; all 32 lanes call it): the rows
// u[r][0][0..V) at columns V*l.., u[r][1][..) at D/2 + V*l.. into codes and pairs, all
// rows' steps side by side.  rows[r]: the row's place in the cache (~0: not written)
// of keys, or (values[r]) of values.
template <int D, int kBits, int R>
__device__ __forceinline__ void put_quantised(const float (&u)[R][2][D / 32], int l, const uint32_t (&rows)[R],
                                              const bool (&values)[R], const abg_kvq_cache &c) {
    constexpr int V = D / 32, C = 2 * R;  // chunks of a lane, 2 r + h
    const int lane = threadIdx.x & 31, group = c.group, log_group = group == 32 ? 5 : 6;
    float lo[C], hi[C];
    const bool joined = group > D / 2;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float &a = lo[2 * r + h], &b = hi[2 * r + h];
            a = INFINITY, b = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) a = least(a, u[r][h][i]), b = largest(b, u[r][h][i]);
        }
        if (joined) {
            lo[2 * r] = lo[2 * r + 1] = least(lo[2 * r], lo[2 * r + 1]);
            hi[2 * r] = hi[2 * r + 1] = largest(hi[2 * r], hi[2 * r + 1]);
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
            lo[i] = least(up ? lo[i + d] : lo[i], a);
            hi[i] = largest(up ? hi[i + d] : hi[i], b);
        }
    }
    for (int d = C; d < lanes; d *= 2) {
        lo[0] = least(lo[0], __shfl_xor_sync(0xffffffffu, lo[0], d));
        hi[0] = largest(hi[0], __shfl_xor_sync(0xffffffffu, hi[0], d));
    }
    constexpr float levels = kBits == 4 ? 15.0f : 255.0f;
    const bool bad = !(hi[0] <= kLargestHalf && lo[0] >= -kLargestHalf);
    const __half nan = __ushort_as_half(0x7fff);
    const __half2 own = bad ? __halves2half2(nan, nan)
                            : __halves2half2(__float2half_rn(__fdiv_rn(__fsub_rn(hi[0], lo[0]), levels)), __float2half_rn(lo[0]));
    const float own_inv = __low2float(own) > 0.0f ? __frcp_rn(__low2float(own)) : 0.0f;  // (a NaN: 0)
    const uint32_t own_pair = *reinterpret_cast<const uint32_t *>(&own);
    const bool first = (l & (lanes - 1)) == 0;  // of a group's lanes
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float x[2][V];
        uint32_t pair[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int from = (lane & ~(C - 1)) + 2 * r + h;
            pair[h] = __shfl_sync(0xffffffffu, own_pair, from);
            const float inv = __shfl_sync(0xffffffffu, own_inv, from);
            const float b = __half2float(__ushort_as_half(static_cast<unsigned short>(pair[h] >> 16)));
            const float2 back = make_float2(-b, -b), times = make_float2(inv, inv), whole = make_float2(12582912.0f, 12582912.0f);
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                // clamped (a NaN to 0), then rounded to a whole number by 1.5 * 2^23
                const float2 y = mul2(add2(make_float2(u[r][h][i], u[r][h][i + 1]), back), times);
                const float2 z = add2(make_float2(fminf(fmaxf(y.x, 0.0f), levels), fminf(fmaxf(y.y, 0.0f), levels)), whole);
                x[h][i] = z.x, x[h][i + 1] = z.y;
            }
        }
        if (rows[r] != ~0u) {
            unsigned char *codes = static_cast<unsigned char *>(values[r] ? c.Vc : c.Kc) +
                                   static_cast<uint64_t>(rows[r]) * (D * kBits / 8) + V * l * kBits / 8;
            store_codes<kBits>(codes, x[0]);
            store_codes<kBits>(codes + D / 2 * kBits / 8, x[1]);
            if (first) {
                uint32_t *pairs = static_cast<uint32_t *>(values[r] ? c.Vs : c.Ks) +
                                  (static_cast<uint64_t>(rows[r]) << (D == 64 ? 6 : D == 128 ? 7 : 8) >> log_group) +
                                  (V * l >> log_group);
                pairs[0] = pair[0];
                if (!joined) pairs[(D / 2) >> log_group] = pair[1];
            }
        }
    }
}

// What the lanes of a warp copy for themselves: `chunks` runs of kBytes a lane, in pieces
// of up to 16 bytes, a piece of all lanes side by side.
template <int kBytes>
struct Pieces {
    static constexpr int kPiece = std::min(kBytes, 16), kParts = kBytes / kPiece;
    __device__ static __forceinline__ void bring(uint32_t to, int chunk, int lane, const void *from) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const uint32_t at = to + (chunk * kParts + i) * 32 * kPiece + lane * kPiece;
            const char *p = static_cast<const char *>(from) + i * kPiece;
            if constexpr (kPiece == 16) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(p) : "memory");
            } else {
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(p), "n"(kPiece) : "memory");
            }
        }
    }
    template <typename S, int V>
    __device__ static __forceinline__ void take(const unsigned char *from, int chunk, int lane, float (&v)[V]) {
        static_assert(V * sizeof(S) == kBytes);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            float t[V / kParts];
            load_e<S, V / kParts>(
                reinterpret_cast<const S *>(from + (chunk * kParts + i) * 32 * kPiece + lane * kPiece), t);
#pragma unroll
            for (int k = 0; k < V / kParts; ++k) v[i * (V / kParts) + k] = t[k];
        }
    }
};

template <typename S, int D>
struct PutRing {  // two units of each warp: their rows and rotations (all warps' first ones, then their second ones)
    static constexpr int V = D / 32;
    using Rows = Pieces<V * sizeof(S)>;
    using Turn = Pieces<V * 4>;
    static constexpr int kRows = 2 * PutUnit<D, false>::kSteps * 32 * V * static_cast<int>(sizeof(S));
    static constexpr int kUnit = kRows + 32 * V * 4;
    static constexpr int kStage = kPutWarps * kUnit;
};

// A warp's way through the units (token n, group of heads g), tokens first.
struct PutWalk {
    uint64_t page_mul;  // 2^64 / page rounded up (page 1: 0): slot / page = page_mul * slot >> 64 for slots below 2^32
    uint32_t dn;        // from one of a warp's units to its next: tokens
    int dg, groups;     // and groups; all groups
};

template <typename S, typename T, int D, int kBits, bool kOnce>
__global__ void __launch_bounds__(32 * kPutWarps, PutUnit<D, kOnce>::kBlocks) kvq_put_kernel(
    const __grid_constant__ abg_kvq_put_args a, const __grid_constant__ PutWalk walk) {
    using P = PutUnit<D, kOnce>;
    using Ring = PutRing<S, D>;
    constexpr int V = P::V, kSteps = P::kSteps;
    extern __shared__ __align__(16) unsigned char raw[];
    const int lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (known to be the same for all lanes)
    unsigned char *ring = raw + warp * Ring::kUnit;
    const int nq = a.q ? static_cast<int>(a.Hq) : 0, nk = static_cast<int>(a.c.Hkv), heads = nq + 2 * nk;
    // (no launch after this one starts early: some read caches and weights before they wait)
    grid_dep_wait();
    struct Token {
        uint32_t n;
        int32_t src;  // -1: none
        int64_t slot;
        int32_t pos;
        int h0;       // first head; below 0: no unit
    };
    // all tokens' last heads (keys and values, the longest work) first, so that every
    // warp has its share of each kind
    const uint32_t N = static_cast<uint32_t>(a.N), unit = blockIdx.x * kPutWarps + warp;
    int g = static_cast<int>(unit / N);
    uint32_t n = unit - g * N;
    auto token = [&] {
        Token t{n, -1, -1, 0, (walk.groups - 1 - g) * P::kHeads};
        if (t.h0 >= 0) {
            t.src = a.rows ? a.rows[n] : static_cast<int32_t>(n);
            if (t.src >= a.src_rows) t.src = -1;
            t.slot = a.slots ? a.slots[n] : n;
            if (a.cos) t.pos = a.pos[n];
        }
        n += walk.dn, g += walk.dg;
        if (n >= N) n -= N, ++g;
        return t;
    };
    // the lane's columns of its head r of a unit; at[r]: of row 0
    const S *at[kSteps];
    int at_h0 = -1;
    auto turn_to = [&](const Token &t) {
        if (t.h0 == at_h0) return;
        at_h0 = t.h0;
#pragma unroll
        for (int r = 0; r < kSteps; ++r) {
            const int h = t.h0 + 2 * r + half;
            at[r] = V * l + (h < nq        ? static_cast<const S *>(a.q) + h * a.q_head
                             : h < nq + nk ? static_cast<const S *>(a.k) + (h - nq) * a.k_head
                                           : static_cast<const S *>(a.v) + min(h - nq - nk, nk - 1) * a.v_head);
        }
    };
    auto source = [&](const Token &t, int r) {  // (past the last head: the last again)
        const int h = t.h0 + 2 * r + half;
        return at[r] + t.src * (h < nq ? a.q_row : h < nq + nk ? a.k_row : a.v_row);
    };
    auto turned = [&](const Token &t) { return t.pos >= 0 && t.pos < a.cos_rows; };
    // a unit's rows and (the lower half's lanes cos, the upper's sin) rotations on their way
    auto bring = [&](const Token &t, int stage) {
        if (t.src >= 0) {
            turn_to(t);
            const uint32_t to = smem_u32(ring) + stage * Ring::kStage;
#pragma unroll
            for (int r = 0; r < kSteps; ++r) {
                const S *p = source(t, r);
                Ring::Rows::bring(to, 2 * r, lane, p);
                Ring::Rows::bring(to, 2 * r + 1, lane, p + D / 2);
            }
            if (a.cos && t.h0 < nq + nk && turned(t))
                Ring::Turn::bring(to + Ring::kRows, 0, lane,
                                  (half ? a.sin : a.cos) + t.pos * static_cast<int64_t>(D / 2) + V * l);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    Token t = token(), next{0, -1, -1, 0, -1};
    if constexpr (!kOnce) next = token();
    if constexpr (!kOnce) bring(t, 0);
    for (int stage = 0; t.h0 >= 0; stage ^= 1) {
        Token after{0, -1, -1, 0, -1};
        if constexpr (!kOnce) {
            __syncwarp();  // the other place has been read
            bring(next, stage ^ 1);
            after = token();
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
        }
        if (t.src >= 0) {
            float u[kSteps][2][V], c[V], s[V];
            const bool turn = a.cos && t.h0 < nq + nk;
            if constexpr (kOnce) {
                turn_to(t);
#pragma unroll
                for (int r = 0; r < kSteps; ++r) {
                    const S *p = source(t, r);
                    load_e<S, V>(p, u[r][0]);
                    load_e<S, V>(p + D / 2, u[r][1]);
                }
                if (turn && turned(t)) {
                    load_e<float, V>(a.cos + t.pos * static_cast<int64_t>(D / 2) + V * l, c);
                    load_e<float, V>(a.sin + t.pos * static_cast<int64_t>(D / 2) + V * l, s);
                }
            } else {
                const unsigned char *from = ring + stage * Ring::kStage;
#pragma unroll
                for (int r = 0; r < kSteps; ++r) {
                    Ring::Rows::template take<S, V>(from, 2 * r, lane, u[r][0]);
                    Ring::Rows::template take<S, V>(from, 2 * r + 1, lane, u[r][1]);
                }
                if (turn) {
                    Ring::Turn::template take<float, V>(from + Ring::kRows, 0, l, c);
                    Ring::Turn::template take<float, V>(from + Ring::kRows, 0, l + 16, s);
                }
            }
            if (turn && !turned(t))
#pragma unroll
                for (int i = 0; i < V; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
            float factor = 0.0f;  // lane r of a half: of the half's head of step r
            if ((a.qn_w && t.h0 < nq) || (a.kn_w && t.h0 < nq + nk && t.h0 + P::kHeads > nq)) {
                float ss = 0.0f;
#pragma unroll
                for (int r = 0; r < kSteps; ++r) {
                    const float lo = square_tree<V>(u[r][0]), hi = square_tree<V>(u[r][1]);
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
            // (a cache has fewer than 2^32 - 1 rows)
            const uint32_t slot = static_cast<uint32_t>(t.slot), page_size = static_cast<uint32_t>(a.c.page);
            const uint64_t low = (walk.page_mul & 0xffffffffu) * slot >> 32, page64 = ((walk.page_mul >> 32) * slot + low) >> 32;
            const uint32_t page = walk.page_mul ? static_cast<uint32_t>(page64) : slot;
            const uint32_t base = page * (nk * page_size) + (slot - page * page_size);
            uint32_t rows[kSteps];
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
                        for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                            for (int i = 0; i < V; i += 2) {
                                const float2 y = mul2(mul2(make_float2(u[r][h2][i], u[r][h2][i + 1]), make_float2(f, f)),
                                                      make_float2(wv[h2][i], wv[h2][i + 1]));
                                u[r][h2][i] = y.x, u[r][h2][i + 1] = y.y;
                            }
                    }
                    if (a.cos) {
#pragma unroll
                        for (int i = 0; i < V; i += 2) {  // (scalar sums: a packed one could be contracted)
                            const float2 x = make_float2(u[r][0][i], u[r][0][i + 1]), y = make_float2(u[r][1][i], u[r][1][i + 1]);
                            const float2 cc = make_float2(c[i], c[i + 1]), ss = make_float2(s[i], s[i + 1]);
                            const float2 xc = mul2(x, cc), ys = mul2(y, ss), yc = mul2(y, cc), xs = mul2(x, ss);
                            u[r][0][i] = __fsub_rn(xc.x, ys.x), u[r][0][i + 1] = __fsub_rn(xc.y, ys.y);
                            u[r][1][i] = __fadd_rn(yc.x, xs.x), u[r][1][i + 1] = __fadd_rn(yc.y, xs.y);
                        }
                    }
                }
                if (h < nq) {
                    T *to = static_cast<T *>(a.qo) + (static_cast<int64_t>(t.n) * nq + h) * D;
                    store_e<T, V>(to + V * l, u[r][0]);
                    store_e<T, V>(to + D / 2 + V * l, u[r][1]);
                }
                values[r] = h >= nq + nk;
                rows[r] = kept && h >= nq && h < heads ? base + (values[r] ? h - nq - nk : h - nq) * page_size : ~0u;
            }
            if (t.h0 + P::kHeads > nq) put_quantised<D, kBits>(u, l, rows, values, a.c);  // (the whole warp, or none of it)
        }
        t = next, next = after;
    }
}

// ------------------------------------------------------------- kvq_get -----
// A thread eight columns of a key or value head, for token after token: one or two words
// and a pair in, 16 or 32 bytes out, so that all but a token's row is known before the
// first.  A block's threads have a token's heads side by side, and as many tokens as there
// is room for; four of a thread's tokens at a time, so that their words are on their way
// together.  Instructions bound it: 32768 tokens of 4 heads of 128, 4 bits to bf16, in
// 17.2 us (86 MB, 5.0 TB/s); with every place found on its own 24.4, with the codes made
// floats by conversions and 64-bit divisions 40.6.
constexpr int kGetThreads = 256, kGetEach = 4, kGetTokens = 128;

// Byte k of w plus 2^23, as a float (0x4b000000 + c).
template <int k>
__device__ __forceinline__ float byte_value(uint32_t w) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + k));
}

// per: places of eight columns of a token (key or value, head, columns); side: tokens side
// by side in a block; tokens: of a block
template <typename T, int kBits>
__global__ void __launch_bounds__(kGetThreads) kvq_get_kernel(const __grid_constant__ abg_kvq_get_args a, int log_cols,
                                                              int per, int side, int tokens) {
    __shared__ uint32_t s_row[kGetTokens];  // of head 0 (a cache has fewer than 2^32 rows); ~0: none
    const int tid = threadIdx.x, Hkv = static_cast<int>(a.c.Hkv), log_pair = a.c.group == 32 ? 2 : 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * tokens;
    const int here = static_cast<int>(min(static_cast<int64_t>(tokens), a.N - n0));
    int first = 0, place = blockIdx.y * kGetThreads + tid;  // the thread's first token, and its place in a token
    if (per < kGetThreads) first = tid / per, place = tid - first * per;
    const int col = place & ((1 << log_cols) - 1), kh = place >> log_cols;
    const bool value = kh >= Hkv || !a.k;
    const int h = kh >= Hkv ? kh - Hkv : kh;
    const int64_t at0 = ((h * a.c.page) << log_cols) + col;
    const uint32_t *codes = static_cast<const uint32_t *>(value ? a.c.Vc : a.c.Kc) + at0 * (kBits / 4);
    const __half2 *pairs = static_cast<const __half2 *>(value ? a.c.Vs : a.c.Ks) + (at0 >> log_pair);
    const int log_words = log_cols + (kBits == 8), log_pairs = log_cols - log_pair;
    const int64_t step = value ? a.v_row : a.k_row;
    T *to = static_cast<T *>(value ? a.v : a.k) + (n0 + first) * step + h * (value ? a.v_head : a.k_head) + 8 * col;
    grid_dep_wait();  // (and nothing after this one starts early, as kvq_put)
    if (tid < here) {
        const int64_t slot = a.slots ? a.slots[n0 + tid] : n0 + tid;
        uint32_t row = ~0u;
        if (slot >= 0 && slot < a.c.pages * a.c.page) {
            const int64_t page = div_up_to_64(slot, a.c.page);
            row = static_cast<uint32_t>(page * Hkv * a.c.page + (slot - page * a.c.page));
        }
        s_row[tid] = row;
    }
    __syncthreads();
    if (first >= side || place >= per) return;
    for (int n = first; n < here; n += kGetEach * side) {
        uint2 w[kGetEach];
        __half2 f[kGetEach];
#pragma unroll
        for (int k = 0; k < kGetEach; ++k) {
            w[k] = make_uint2(0, 0);
            f[k] = __float2half2_rn(0.0f);
            if (n + k * side >= here) continue;
            const uint32_t row = s_row[n + k * side];
            if (row == ~0u) continue;
            const uint32_t *from = codes + (static_cast<uint64_t>(row) << log_words);
            if constexpr (kBits == 4) {
                w[k].x = *from;
            } else {
                w[k] = *reinterpret_cast<const uint2 *>(from);
            }
            f[k] = pairs[static_cast<uint64_t>(row) << log_pairs];
        }
#pragma unroll
        for (int k = 0; k < kGetEach; ++k) {
            if (n + k * side >= here) continue;
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
            const float2 sb = __half22float2(f[k]);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {  // (the product is exact: 11 and 8 bits)
                const float2 y = fma2(make_float2(sb.x, sb.x), add2(make_float2(v[i], v[i + 1]), make_float2(-8388608.0f, -8388608.0f)),
                                      make_float2(sb.y, sb.y));
                v[i] = y.x, v[i + 1] = y.y;
            }
            store_e<T, 8>(to, v);
            to += side * step;
        }
    }
}

// kOnce: false if the call is too long for it
template <typename S, typename T, int D, int kBits, bool kOnce>
bool put_units(const abg_kvq_put_args &a, bool early, cudaStream_t stream, cudaError_t &e) {
    constexpr int kSmem = kOnce ? 0 : 2 * PutRing<S, D>::kStage, kHeads = PutUnit<D, kOnce>::kHeads;
    const auto kernel = kvq_put_kernel<S, T, D, kBits, kOnce>;
    static const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (attr != cudaSuccess) {
        e = attr;
        return true;
    }
    // as many blocks as fit at once
    static const int fit = [&] {
        int per = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, 32 * kPutWarps, kSmem) != cudaSuccess) per = 1;
        return std::max(per, 1) * sm_count();
    }();
    const int heads = static_cast<int>((a.q ? a.Hq : 0) + 2 * a.c.Hkv), groups = (heads + kHeads - 1) / kHeads;
    const int64_t blocks = (a.N * groups + kPutWarps - 1) / kPutWarps;
    if (kOnce && blocks > fit) return false;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, fit));
    const uint64_t stride = uint64_t(grid) * kPutWarps, N = static_cast<uint64_t>(a.N), page = static_cast<uint64_t>(a.c.page);
    const PutWalk walk{page == 1 ? 0 : ~uint64_t(0) / page + 1, static_cast<uint32_t>(stride % N), static_cast<int>(stride / N),
                       groups};
    e = launch_kernel(kernel, dim3(grid), dim3(32 * kPutWarps), kSmem, stream, early, a, walk);
    return true;
}
template <typename S, typename T, int D, int kBits>
cudaError_t put_d(const abg_kvq_put_args &a, bool early, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (!put_units<S, T, D, kBits, true>(a, early, stream, e)) put_units<S, T, D, kBits, false>(a, early, stream, e);
    return e;
}
template <typename S, typename T, int kBits>
cudaError_t put_bits(const abg_kvq_put_args &a, bool early, cudaStream_t stream) {
    return a.c.D == 64    ? put_d<S, T, 64, kBits>(a, early, stream)
           : a.c.D == 128 ? put_d<S, T, 128, kBits>(a, early, stream)
                          : put_d<S, T, 256, kBits>(a, early, stream);
}
template <typename S, typename T>
cudaError_t put(const abg_kvq_put_args &a, bool early, cudaStream_t stream) {
    return a.c.bits == 4 ? put_bits<S, T, 4>(a, early, stream) : put_bits<S, T, 8>(a, early, stream);
}

template <typename T, int kBits>
cudaError_t get_bits(const abg_kvq_get_args &a, bool pdl, cudaStream_t stream) {
    const int kinds = (a.k != nullptr) + (a.v != nullptr);
    const int log_cols = a.c.D == 64 ? 3 : a.c.D == 128 ? 4 : 5;
    const int per = kinds * static_cast<int>(a.c.Hkv) << log_cols;
    const int side = std::min(std::max(1, kGetThreads / per), kGetTokens / 8), parts = (per + kGetThreads - 1) / kGetThreads;
    // eight tokens a thread, as long as there are eight blocks an SM
    const int64_t each = std::max<int64_t>(1, std::min<int64_t>(8, a.N * parts / side / (8ll * sm_count())));
    const int64_t tokens = each * side;
    return launch_kernel(kvq_get_kernel<T, kBits>,
                         dim3(static_cast<unsigned>((a.N + tokens - 1) / tokens), static_cast<unsigned>(parts)),
                         dim3(kGetThreads), 0, stream, pdl && !capturing(stream), a, log_cols, per, side,
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
