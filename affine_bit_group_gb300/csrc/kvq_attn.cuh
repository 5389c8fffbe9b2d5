// kvq_attn: attention of new tokens over a quantised paged cache and over one
// another (formulas in include/abg.h, the work split in tree_attn.cuh).
//
// Mathematics.  A cached K row is k_i = s_g c_i + b_g in groups g of 32 or 64
// columns, so
//     q.k = sum_g ( s_g sum_i q_i c_i + b_g sum_i q_i ),
// the weights' own formula (y = scale * (codes . x) + bias * group sum of x), and
//     sum_t p_t v_ti = sum_t (p_t s_tg) c_ti + sum_t p_t b_tg.
// The codes never become values: they are the tensor cores' operands as they are.
// A code c under the mask 0x000f000f (4 bits) or 0x00ff00ff (8) is the f16 number
// c * 2^-24, a subnormal, and a nibble left where it is under 0x00f000f0 is c *
// 2^-20; the powers of two go into q and into the results.  Taking eight 4-bit codes
// apart is then five integer instructions.  The tensor cores line the products up by
// the factors' exponents, though, and a subnormal's is that of 2^-14: sums of such
// products keep fewer bits, which bf16 results do not show and f32 ones do (2.7e-4
// relative).  With f16 and f32 queries the codes are therefore made normal numbers
// around 0, one more instruction for two: K's as c - 8 or c - 128, V's as c - z with z =
// -b/s of the token and group rounded to a code, which leaves at most s/2 of b.  (Codes
// from 0 on leave the two sums of V large and of opposite signs where the values
// themselves cancel: 1e-5 relative over 2000 tokens.  From the middle on they do so
// where values are one-sided: a token of nearly all weight and a V of 0 would push the
// others' small parts out of the 24 bits.)  The products' sums of a block meet those of
// the blocks before in f32 that rounds to nearest, since the tensor cores cut off.
//
// Tiles.  K and V are the products' first operand (16 tokens of K by 16 columns,
// 16 columns of V by 16 tokens) and the query rows, 8 at a time, their second: one
// new token of a request has Hq/Hkv rows, 1 to 8 or so, which would leave most of a
// 64- or 128-row tile of the tcgen05 products empty, whose operands would also have
// to go through shared memory as 16-bit values, four times the bytes of the cache
// (mma.sync takes them from registers).  What the lanes load is chosen so that a
// lane's words hold the columns and tokens that its places in the products ask for;
// the weights P go from the one product's result to the other's operand by
// movmatrix, in registers.
//
// Warps.  Every warp goes through blocks of 16 or 32 tokens of its own (block w, w +
// 8, .. of the stretch), with a ring in shared memory that it fills by cp.async and
// its own running maxima and sums: no barrier until the stretch's end, where the
// warps' sums meet in shared memory, and the drafts are added, in f32, a row a warp.
#pragma once

#include "kv_rows.cuh"
#include "kvq.cuh"
#include "tree_attn.cuh"

#include <algorithm>

namespace abg {

struct KvqAttnArgs {
    AttnArgs p;
    const unsigned char *Kc, *Vc;
    const unsigned char *Ks, *Vs;
    uint32_t page_mul;  // t / page = (t * page_mul >> 32) >> page_shift for t < 2^31 (0: page 1)
    int page_shift;
};

// The multiplier of a division by page: 2^(31 + s) / page rounded up, where 2^s is the
// power of two from page on, is off by less than 1 part in 2^31.
inline void kvq_page_division(KvqAttnArgs &x, uint32_t page) {
    int s = 0;
    while (s < 31 && (1u << s) < page) ++s;
    x.page_mul = page == 1 ? 0 : static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + page - 1) / page);
    x.page_shift = s - 1;
}

constexpr int kKvqWarps = 8, kKvqThreads = 32 * kKvqWarps;
constexpr int kKvqTile = 128;  // tokens of the work line's tiles
// Rows of q from here on give NaN: their scores could pass f32's range.
constexpr float kKvqLargestQ = 1.2676506e30f;  // 2^100

template <int D_, int kBits_, int kGroup_, int kNT_, bool kSplit_>
struct KvqShape {
    static constexpr int D = D_, kBits = kBits_, kGroup = kGroup_;
    static constexpr int kNT = kNT_;                      // query rows, by 8
    static constexpr int kTerms = kSplit_ ? 2 : 1;        // f16 terms of q and of P
    // two terms: codes as normal numbers around 0 (K's c - kMiddle, V's c - z), a block's
    // products summed on their own; else codes as subnormal numbers, one sum
    static constexpr bool kNormal = kSplit_;
    static constexpr float kMiddle = kNormal ? (kBits == 4 ? 8.0f : 128.0f) : 0.0f;
    static constexpr float kUnit = kNormal ? 1.0f : 16777216.0f;             // 1 / the operand's value of a code 1
    static constexpr float kUpper = !kNormal && kBits == 4 ? 16.0f : 1.0f;   // an upper nibble's over a lower's
    static constexpr int kRT = 8 * kNT;
    static constexpr int kRB = D * kBits / 8;             // bytes of a row's codes
    static constexpr int kG = D / kGroup, kFB = 4 * kG;   // groups of a row, bytes of its factors
    static constexpr int kTB = kRB <= 64 ? 32 : 16;       // tokens of a block
    static constexpr int kMT = kTB / 16;
    static constexpr int kSteps = D / 16;                 // products of 16 columns
    static constexpr int kWords = kGroup * kBits / 128;   // words of a group in a lane
    // blocks an SM: what the registers (D/4 of sums a row tile) and the ring leave room for
    static constexpr int kBlocks = kNT * D / 4 > 64 || kRB == 256 ? 1 : 2;
    static constexpr int kStageBytes = kTB * 2 * (kRB + kFB);
    static constexpr int kQBytes = kSteps * kTerms * kNT * 32 * 8;
    static constexpr int kZBytes = kNormal ? kTB * kG * 6 : 0;  // a warp's V tokens: f32 rest, f16 -(1024 + z)
    static constexpr int kFixed = kQBytes + 4 * kRT * (kG + 1 + 2 * kKvqWarps) + kKvqWarps * kZBytes;
    static constexpr int kRoom = (kBlocks == 2 ? 113 : 226) * 1024 - kFixed - 1024;
    static constexpr int kStages = std::min(6, kRoom / (kKvqWarps * kStageBytes));
    static constexpr int kRowPair = 2 * D + 2;            // floats of two rows of a warp's sums
    static constexpr int kWarpBytes = std::max(kStages * kStageBytes, kRT / 2 * kRowPair * 4 + 8) / 16 * 16;
    static_assert(kStages >= 2 && kWarpBytes * kKvqWarps <= kRoom, "the ring fits");
    static constexpr int kSmem = kFixed + kKvqWarps * kWarpBytes;
};

// N bytes to shared memory; without kWhole, zeros where they are not real
template <int N, bool kWhole>
__device__ __forceinline__ void kvq_cp(uint32_t dst, const void *src, bool real) {
    if constexpr (kWhole && N == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    } else if constexpr (kWhole) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
    } else if constexpr (N == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(real ? N : 0)
                     : "memory");
    }
}
// 2^x by the special function unit; results below 2^-126 are 0
__device__ __forceinline__ float kvq_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void kvq_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void kvq_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d (16x8, f32) += a (16x16) b (16x8), f16
__device__ __forceinline__ void kvq_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ uint32_t kvq_transpose(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// The two lower or (kUp) upper fields of v's halves, 4 or 8 bits, as f16 operands; where
// these are normal numbers, plus `from` (the lower field's; -1024 - what the codes are
// counted from), since 0x6400 + c is 1024 + c in f16.
template <typename S, bool kUp>
__device__ __forceinline__ uint32_t kvq_operand(uint32_t v, __half2 from) {
    constexpr uint32_t kMask = S::kBits == 8 ? 0x00ff00ffu : kUp ? 0x00f000f0u : 0x000f000fu;
    const uint32_t c = (S::kBits == 8 && kUp ? v >> 8 : v) & kMask;
    if constexpr (S::kNormal) {
        const uint32_t h = c | 0x64006400u;
        __half2 r;
        if constexpr (S::kBits == 4 && kUp) {  // 1024 + 16 c
            r = __hfma2(*reinterpret_cast<const __half2 *>(&h), __float2half2_rn(0.0625f), __hadd2(from, __float2half2_rn(960.0f)));
        } else {
            r = __hadd2(*reinterpret_cast<const __half2 *>(&h), from);
        }
        return *reinterpret_cast<const uint32_t *>(&r);
    } else {
        return c;
    }
}
__device__ __forceinline__ uint32_t kvq_half2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 kvq_float2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// The token of row i of 8 in a 16-token tile (the other 8 rows: 8 more): rows 2c and
// 2c + 1 are tokens c and c + 4, so that the four lanes of a column of V read four
// tokens in a row.
__device__ __forceinline__ int kvq_token(int i) { return (i >> 1) + 4 * (i & 1); }

// Which 16-byte place of a row of the ring a chunk lies in: the rows of one load in
// different banks (counted over all 32 lanes of every load of both products: no
// conflicts left, but for 8 bits in groups of 64 of a 64-column row, 24 for 16).
template <typename S>
__device__ __forceinline__ int kvq_swizzle(int t) {
    constexpr bool narrow = S::kGroup == 32 && S::kBits == 4;
    const int t0 = t & 1, t1 = t >> 1 & 1, t2 = t >> 2 & 1;
    if constexpr (S::kRB == 32) {
        return narrow ? t2 : 0;
    } else if constexpr (S::kRB == 64) {
        return narrow ? t1 + 2 * t2 : S::kBits == 8 && S::kGroup == 64 ? 2 * t1 : 2 * (t1 ^ t2);
    } else {
        return narrow ? t0 + 2 * t1 + 4 * t2 : (2 * t0) ^ (4 * (t1 ^ t2));
    }
}

// E consecutive values of a row of `type`
template <int E>
__device__ __forceinline__ void kvq_row(const void *p, int type, int64_t at, float (&v)[E]) {
    if (type == ABG_SB_F32) {
        load_e<float, E>(static_cast<const float *>(p) + at, v);
    } else if (type == ABG_SB_BF16) {
        load_e<__nv_bfloat16, E>(static_cast<const __nv_bfloat16 *>(p) + at, v);
    } else {
        load_e<__half, E>(static_cast<const __half *>(p) + at, v);
    }
}
__device__ __forceinline__ float kvq_value(const void *p, int type, int64_t at) {
    return type == ABG_SB_F32    ? static_cast<const float *>(p)[at]
           : type == ABG_SB_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at])
                                 : __half2float(static_cast<const __half *>(p)[at]);
}

template <typename S>
__global__ void __launch_bounds__(kKvqThreads, S::kBlocks) kvq_attn_kernel(const __grid_constant__ KvqAttnArgs x) {
    constexpr int D = S::D, kNT = S::kNT, kRT = S::kRT, kRB = S::kRB, kFB = S::kFB, kG = S::kG, kTB = S::kTB;
    constexpr int kMT = S::kMT, kTerms = S::kTerms, kStages = S::kStages, kGroup = S::kGroup, kBits = S::kBits;
    constexpr int E = D / 32, kTiles = D / 16;
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ AttnScan scan;
    const AttnArgs &p = x.p;
    const abg_tree_attn_args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j = lane >> 2, quad = lane & 3;
    uint2 *s_q = reinterpret_cast<uint2 *>(raw);                            // [step][term][row tile][lane]
    float *s_qs = reinterpret_cast<float *>(raw + S::kQBytes);              // [kG][kRT] group sums of q
    float *s_f = s_qs + kG * kRT;                                           // [kRT] factor of a row's scores
    float *s_m = s_f + kRT, *s_l = s_m + kKvqWarps * kRT;                   // [warp][kRT]
    float *rest = reinterpret_cast<float *>(s_l + kKvqWarps * kRT) + warp * (S::kZBytes / 4);  // [kTB][kG]
    __half *zero = reinterpret_cast<__half *>(rest + kTB * kG);                               // [kG][kTB], pairs
    unsigned char *ring = raw + (S::kFixed + warp * S::kWarpBytes);
    const uint32_t ring_at = smem_u32(ring);
    static_assert(S::kFixed % 16 == 0, "the ring's alignment");
    grid_dep_wait();
    grid_dep_launch();
    AttnLine<kRT, kKvqTile> line;
    line.template init<kKvqThreads>(p, blockIdx.x, gridDim.x, scan);
    bool left = false;
    AttnSeg s;
    while (line.next(p, s)) {
        const int key0 = min(s.t0, s.ctiles) * kKvqTile;
        const int key1 = min(s.req.len, min(s.t1, s.ctiles) * kKvqTile);    // cached tokens of the stretch
        const int blocks = key1 > key0 ? (key1 - key0 + kTB - 1) / kTB : 0;
        // -- copies --
        const int32_t *table = a.table + static_cast<int64_t>(s.b) * a.width;
        auto page_at = [&](int t) {
            return x.page_mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(t), x.page_mul) >> x.page_shift) : t;
        };
        auto page_of = [&](int blk) {  // of this lane's token
            const int t = key0 + blk * kTB + lane;
            return blk < blocks && lane < kTB && t < key1 ? table[page_at(t)] : -1;
        };
        int32_t id = page_of(warp);
        auto bring = [&](int i) {  // the warp's block i, of whose pages `id` knows; a group of copies
            const int blk = warp + i * kKvqWarps;
            if (blk < blocks) {
                const int t = key0 + blk * kTB + lane, page = static_cast<int>(a.page);
                const bool there = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.pages);
                // (a cache has fewer than 2^32 rows)
                const uint32_t row =
                    there ? (static_cast<uint32_t>(id) * static_cast<uint32_t>(a.Hkv) + s.h) * page + (t - page_at(t) * page) : 0;
                id = page_of(blk + kKvqWarps);
                const uint32_t at = ring_at + (i % kStages) * S::kStageBytes;
                constexpr int kChunks = kRB / 16;
                const unsigned all = __ballot_sync(0xffffffffu, there);
                auto copy = [&](auto whole) {
                    constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
                    for (int c = 0; c < kTB * kChunks / 32; ++c) {
                        const int tok = 32 / kChunks * c + lane / kChunks, ch = lane % kChunks;
                        const int64_t off = static_cast<uint64_t>(__shfl_sync(0xffffffffu, row, tok)) * kRB + 16 * ch;
                        const uint32_t to = at + tok * kRB + 16 * (ch ^ kvq_swizzle<S>(tok));
                        const bool real = kWhole || (all >> tok & 1);
                        kvq_cp<16, kWhole>(to, x.Kc + off, real);
                        kvq_cp<16, kWhole>(to + kTB * kRB, x.Vc + off, real);
                    }
                    if (lane < kTB) {
                        constexpr int kEach = kFB < 16 ? kFB : 16;
                        const uint32_t to = at + 2 * kTB * kRB + lane * kFB;
                        const int64_t off = static_cast<uint64_t>(row) * kFB;
#pragma unroll
                        for (int c = 0; c < kFB; c += kEach) {
                            kvq_cp<kEach, kWhole>(to + c, x.Ks + off + c, there);
                            kvq_cp<kEach, kWhole>(to + kTB * kFB + c, x.Vs + off + c, there);
                        }
                    }
                };
                constexpr unsigned kAll = kTB == 32 ? 0xffffffffu : 0xffffu;
                if ((all & kAll) == kAll) {
                    copy(std::true_type{});
                } else {  // a last block, or pages that there are not: zeros
                    copy(std::false_type{});
                }
            }
            kvq_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) bring(i);
        // -- q: a row a warp for its scale and sums, then the products' operands --
        if (blocks > 0) {
            for (int r = warp; r < kRT; r += kKvqWarps) {
                float v[E];
                const int q = s.r0 + r;
                float top = 0.0f;
                if (r < s.rows) {
                    kvq_row<E>(a.q, a.type, ((static_cast<int64_t>(s.req.n0) + q / p.G) * a.Hq + s.h * p.G + q % p.G) * D + lane * E, v);
                } else {
#pragma unroll
                    for (int i = 0; i < E; ++i) v[i] = 0.0f;
                }
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    top = fabsf(v[i]) < INFINITY ? fmaxf(top, fabsf(v[i])) : INFINITY;
                    sum += v[i];
                }
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
                for (int d = kGroup / E / 2; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                // the row's largest in 2^13 .. 2^14 (below 2^-87: lower)
                const int ex = min(100, 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127));
                const bool bad = top >= kKvqLargestQ, none = top == 0.0f;
                const float up = bad || none ? 1.0f : pow2i(ex);
                // s_f * (s acc + b qs) is the score in base 2, acc of the scaled q and the operands
                if (lane == 0) s_f[r] = bad ? __int_as_float(0x7fc00000) : p.scale2 * S::kUnit / up;
                if (lane % (kGroup / E) == 0) s_qs[lane / (kGroup / E) * kRT + r] = sum * up * (1.0f / S::kUnit);
                if (lane == 1) s_l[r] = up;  // (until the operands are made)
            }
            __syncthreads();
            for (int i = tid; i < S::kSteps * kNT * 32; i += kKvqThreads) {
                const int ln = i & 31, nt = i / 32 % kNT, step = i / (32 * kNT);
                const int r = nt * 8 + (ln >> 2), q = s.r0 + r;
                constexpr int kPerWord = kBits == 4 ? 2 : 1;  // steps of a word
                const int w = step / kPerWord, g = w / S::kWords, wi = w % S::kWords;
                const int col = g * kGroup + ((ln & 3) * S::kWords + wi) * (32 / kBits) + (kBits == 4 ? 2 * (step % 2) : 0);
                float v[4] = {};
                if (r < s.rows) {
                    const int64_t at = ((static_cast<int64_t>(s.req.n0) + q / p.G) * a.Hq + s.h * p.G + q % p.G) * D + col;
                    const float up = s_l[r];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // the pairs' columns: 0 and 4, 1 and 5 of 4 bits (the second a nibble
                        // up: 2^4), 0 and 2, 1 and 3 of 8
                        const float t = kvq_value(a.q, a.type, at + (k >> 1) + (k & 1) * (kBits == 4 ? 4 : 2)) * up;
                        v[k] = k >> 1 ? t * (1.0f / S::kUpper) : t;
                    }
                }
                uint2 *to = s_q + ((step * kTerms) * kNT + nt) * 32 + ln;
                const uint2 hi = make_uint2(kvq_half2(v[0], v[1]), kvq_half2(v[2], v[3]));
                *to = hi;
                if constexpr (kTerms == 2) {
                    const float2 h0 = kvq_float2(hi.x), h1 = kvq_float2(hi.y);
                    to[kNT * 32] = make_uint2(kvq_half2(v[0] - h0.x, v[1] - h0.y), kvq_half2(v[2] - h1.x, v[3] - h1.y));
                }
            }
            __syncthreads();
        }
        // -- the warp's blocks --
        float o[kTiles][kNT][4];             // columns (8 or 4 a lane of a group, two a tile) x rows 2 quad, + 1
        float l[kNT][2], m[kNT][2], bias[kG][kNT][2];
        int ev = 0;                          // the largest scale of V so far is below 2^(ev - 14)
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            l[nt][0] = l[nt][1] = 0.0f;
            m[nt][0] = m[nt][1] = -INFINITY;
#pragma unroll
            for (int g = 0; g < kG; ++g) bias[g][nt][0] = bias[g][nt][1] = 0.0f;
        }
        const int tok = kvq_token(j);
        for (int i = 0, blk = warp; blk < blocks; ++i, blk += kKvqWarps) {
            kvq_wait<kStages - 2>();
            __syncwarp();  // every lane's copies have come, and the last block's place is free
            bring(i + kStages - 1);
            const unsigned char *K = ring + (i % kStages) * S::kStageBytes, *V = K + kTB * kRB, *Kf = V + kTB * kRB,
                                *Vf = Kf + kTB * kFB;
            // scores
            float sc[kMT][kNT][4];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.0f;
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                uint32_t w[kMT][2][S::kWords];
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int off = g * (kGroup * kBits / 8) + quad * (4 * S::kWords);
                        const unsigned char *from =
                            K + (16 * mt + 8 * h + tok) * kRB + (((off >> 4) ^ kvq_swizzle<S>(tok)) << 4) + (off & 15);
                        if constexpr (S::kWords == 1) {
                            w[mt][h][0] = *reinterpret_cast<const uint32_t *>(from);
                        } else if constexpr (S::kWords == 2) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(from);
                            w[mt][h][0] = v.x, w[mt][h][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4 *>(from);
                            w[mt][h][0] = v.x, w[mt][h][1] = v.y, w[mt][h][2] = v.z, w[mt][h][3] = v.w;
                        }
                    }
                float acc[kMT][kNT][4];
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.0f;
                constexpr int kPerWord = kBits == 4 ? 2 : 1;
#pragma unroll
                for (int wi = 0; wi < S::kWords; ++wi)
#pragma unroll
                    for (int hh = 0; hh < kPerWord; ++hh) {
                        const int step = (g * S::kWords + wi) * kPerWord + hh;
                        uint32_t e[kMT][4];
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t v = w[mt][h][wi] >> (8 * hh);
                                const __half2 from = __float2half2_rn(-1024.0f - S::kMiddle);
                                e[mt][h] = kvq_operand<S, false>(v, from);
                                e[mt][2 + h] = kvq_operand<S, true>(v, from);
                            }
#pragma unroll
                        for (int term = 0; term < kTerms; ++term)
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt) {
                                const uint2 b = s_q[((step * kTerms + term) * kNT + nt) * 32 + lane];
#pragma unroll
                                for (int mt = 0; mt < kMT; ++mt)
                                    kvq_mma(acc[mt][nt], e[mt][0], e[mt][1], e[mt][2], e[mt][3], b);
                            }
                    }
                float2 f[kMT][2];  // scale, bias of tokens tok and tok + 8
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f[mt][h] = kvq_float2(*reinterpret_cast<const uint32_t *>(Kf + (16 * mt + 8 * h + tok) * kFB + 4 * g));
                        if constexpr (S::kNormal) f[mt][h].y = fmaf(S::kMiddle, f[mt][h].x, f[mt][h].y);
                    }
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    const float2 qs = *reinterpret_cast<const float2 *>(s_qs + g * kRT + nt * 8 + 2 * quad);
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[mt][nt][e] = fmaf(acc[mt][nt][e], f[mt][e >> 1].x,
                                                 g == 0 ? f[mt][e >> 1].y * (e & 1 ? qs.y : qs.x)
                                                        : fmaf(f[mt][e >> 1].y, e & 1 ? qs.y : qs.x, sc[mt][nt][e]));
                }
            }
            // maxima and weights (sc is in units of 1/s_f until its exponential)
            const int here = key1 - key0 - blk * kTB;  // tokens of the block that are there
            if (here < kTB) {
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (16 * mt + 8 * (e >> 1) + tok >= here) sc[mt][nt][e] = -INFINITY;
            }
            bool grew = false;
            float corr[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const float2 f = *reinterpret_cast<const float2 *>(s_f + nt * 8 + 2 * quad);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(sc[0][nt][e], sc[0][nt][2 + e]);
                    if constexpr (kMT == 2) top = fmaxf(top, fmaxf(sc[kMT - 1][nt][e], sc[kMT - 1][nt][2 + e]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    top = fmaxf(m[nt][e], top * (e ? f.y : f.x));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    corr[nt][e] = kvq_exp2(m[nt][e] - ref);
                    grew = grew || top > m[nt][e];
                    m[nt][e] = top;
                    float sum = 0.0f;
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float &v = sc[mt][nt][2 * h + e];
                            v = kvq_exp2(fmaf(v, e ? f.y : f.x, -ref));
                            sum += v;
                        }
                    l[nt][e] = fmaf(l[nt][e], corr[nt][e], sum);
                }
            }
            // the largest scale of V
            uint32_t big = 0;
            if (lane < kTB) {
#pragma unroll
                for (int g = 0; g < kG; ++g) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(Vf + lane * kFB + 4 * g), v = w & 0x7fffu;
                    big = max(big, v < 0x7c00u ? v : 0u);
                    if constexpr (S::kNormal) {
                        const float2 f = kvq_float2(w);
                        // (any z is right; no scale, or a NaN: one of the ends)
                        const float z = fminf(fmaxf(rintf(__fdividef(-f.y, f.x)), 0.0f), kBits == 4 ? 15.0f : 255.0f);
                        rest[lane * kG + g] = fmaf(f.x, z, f.y);
                        zero[g * kTB + (lane & ~7) + 2 * (lane & 3) + (lane >> 2 & 1)] = __float2half_rn(-1024.0f - z);
                    }
                }
            }
            const int ev0 = static_cast<int>(__reduce_max_sync(0xffffffffu, big) >> 10), ev1 = S::kNormal ? ev0 : max(ev, ev0);
            if constexpr (S::kNormal) __syncwarp();
            if (__any_sync(0xffffffffu, grew) || (!S::kNormal && ev1 != ev)) {
                const float down = S::kNormal ? 1.0f : pow2i(ev - ev1);
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                    for (int g = 0; g < kG; ++g) bias[g][nt][0] *= corr[nt][0], bias[g][nt][1] *= corr[nt][1];
                    const float c0 = corr[nt][0] * down, c1 = corr[nt][1] * down;
#pragma unroll
                    for (int i = 0; i < kTiles; ++i)
                        o[i][nt][0] *= c0, o[i][nt][1] *= c1, o[i][nt][2] *= c0, o[i][nt][3] *= c1;
                }
            }
            ev = ev1;
            const float up = pow2i(28 - ev);
            // weighted sums
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                constexpr int kPart = S::kNormal ? kGroup / 16 : 1;
                float part[kPart][kNT][4];  // of the block
                if constexpr (S::kNormal) {
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                        for (int i = 0; i < kPart; ++i) part[i][nt][0] = part[i][nt][1] = part[i][nt][2] = part[i][nt][3] = 0.0f;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
                    float2 f[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f[h] = kvq_float2(*reinterpret_cast<const uint32_t *>(Vf + (16 * mt + 8 * h + tok) * kFB + 4 * g));
                        if constexpr (S::kNormal) f[h].y = rest[(16 * mt + 8 * h + tok) * kG + g];
                        f[h].x *= up;
                    }
                    uint2 b[kTerms][kNT];
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
                        const float *w = sc[mt][nt];
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[e] = w[e] * f[e >> 1].x;
                            bias[g][nt][e & 1] = fmaf(w[e], f[e >> 1].y, bias[g][nt][e & 1]);
                        }
                        const uint32_t h0 = kvq_half2(v[0], v[1]), h1 = kvq_half2(v[2], v[3]);
                        b[0][nt] = make_uint2(kvq_transpose(h0), kvq_transpose(h1));
                        if constexpr (kTerms == 2) {
                            const float2 r0 = kvq_float2(h0), r1 = kvq_float2(h1);
                            b[1][nt] = make_uint2(kvq_transpose(kvq_half2(v[0] - r0.x, v[1] - r0.y)),
                                                  kvq_transpose(kvq_half2(v[2] - r1.x, v[3] - r1.y)));
                        }
                    }
                    __half2 z[2];  // of tokens quad and + 4, + 8 and + 12
                    if constexpr (S::kNormal) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            z[k] = *reinterpret_cast<const __half2 *>(zero + g * kTB + 16 * mt + 8 * k + 2 * quad);
                    }
                    // the lane's columns of the group, of those tokens
                    constexpr int kCols = kGroup / 8;
                    uint32_t u[4][kCols * kBits / 32 > 0 ? kCols * kBits / 32 : 1];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int t = quad + 4 * k;
                        const int off = g * (kGroup * kBits / 8) + (kCols * kBits / 8 * j & ~3);
                        const unsigned char *from =
                            V + (16 * mt + t) * kRB + (((off >> 4) ^ kvq_swizzle<S>(t)) << 4) + (off & 15);
                        if constexpr (kCols * kBits == 64) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(from);
                            u[k][0] = v.x, u[k][1] = v.y;
                        } else {
                            u[k][0] = *reinterpret_cast<const uint32_t *>(from);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kGroup / 16; ++i) {  // columns 2 i and 2 i + 1 of the lane's
                        uint32_t e[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {  // tokens quad and + 4, then + 8 and + 12
                            if constexpr (kBits == 4) {
                                // four columns of both tokens
                                const uint32_t pick = kGroup == 32 ? (j & 1 ? 0x7632u : 0x5410u) : i >= 2 ? 0x7632u : 0x5410u;
                                const uint32_t v = __byte_perm(u[2 * k][0], u[2 * k + 1][0], pick) >> (8 * (i % 2));
                                e[2 * k] = kvq_operand<S, false>(v, z[k]), e[2 * k + 1] = kvq_operand<S, true>(v, z[k]);
                            } else {
                                const uint32_t v = __byte_perm(u[2 * k][i / 2], u[2 * k + 1][i / 2], i % 2 ? 0x7632u : 0x5410u);
                                e[2 * k] = kvq_operand<S, false>(v, z[k]), e[2 * k + 1] = kvq_operand<S, true>(v, z[k]);
                            }
                        }
#pragma unroll
                        for (int term = 0; term < kTerms; ++term)
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt)
                                kvq_mma(S::kNormal ? part[S::kNormal ? i : 0][nt] : o[g * (kGroup / 16) + i][nt], e[0], e[1],
                                        e[2], e[3], b[term][nt]);
                    }
                }
                if constexpr (S::kNormal) {
                    const float down = pow2i(ev - 28);
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                        for (int i = 0; i < kPart; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[g * (kGroup / 16) + i][nt][e] = fmaf(part[i][nt][e], down, o[g * (kGroup / 16) + i][nt][e]);
                    }
                }
            }
        }
        kvq_wait<0>();
        __syncwarp();
        // -- the warp's sums to shared memory, in its ring --
        if (blocks > 0) {
            float *mine = reinterpret_cast<float *>(ring);
            const float up = S::kNormal ? 1.0f : pow2i(ev - 28) * S::kUnit;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
#pragma unroll
                        for (int g = 0; g < kG; ++g) bias[g][nt][e] += __shfl_xor_sync(0xffffffffu, bias[g][nt][e], d);
                    }
                    if (j == 0) {
                        s_m[warp * kRT + nt * 8 + 2 * quad + e] = m[nt][e];
                        s_l[warp * kRT + nt * 8 + 2 * quad + e] = l[nt][e];
                    }
                }
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    constexpr int kPer = kGroup / 16;
                    const int g = i / kPer, col = g * kGroup + (kGroup / 8) * j + 2 * (i % kPer);
                    constexpr float kOdd = 1.0f / S::kUpper;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float2 *>(mine + (nt * 4 + quad) * S::kRowPair + e * D + col) =
                            make_float2(fmaf(o[i][nt][e], up, bias[g][nt][e]),
                                        fmaf(o[i][nt][2 + e] * kOdd, up, bias[g][nt][e]));
                }
            }
        }
        __syncthreads();
        // -- a row a warp: the warps' sums, the drafts, the result --
        const bool whole = s.t0 == 0 && s.t1 == s.tiles;
        const int64_t slot = static_cast<int64_t>(2) * blockIdx.x + (s.t0 == 0);
        const int d0 = (max(s.t0, s.ctiles) - s.ctiles) * kKvqTile, d1 = min(s.req.T, (s.t1 - s.ctiles) * kKvqTile);
        for (int r = warp; r < s.rows; r += kKvqWarps) {
            const int q = s.r0 + r, draft = q / p.G, hq = s.h * p.G + q % p.G;
            const int64_t n = static_cast<int64_t>(s.req.n0) + draft;
            float M = -INFINITY, L = 0.0f, v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = 0.0f;
            if (blocks > 0) {
                const int w = lane & 7;
                const float mw = s_m[w * kRT + r], lw = s_l[w * kRT + r];
                M = mw;
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
                // (no maximum, but a weight: a NaN, which stays)
                const float fw = lw == 0.0f ? 0.0f : mw == -INFINITY ? 1.0f : exp2f(mw - M);
#pragma unroll
                for (int u = 0; u < kKvqWarps; ++u) {
                    const float f = __shfl_sync(0xffffffffu, fw, u), lu = __shfl_sync(0xffffffffu, lw, u);
                    if (f == 0.0f) continue;  // no weight: nothing to add
                    L = fmaf(lu, f, L);
                    const float *from = reinterpret_cast<const float *>(raw + S::kFixed + u * S::kWarpBytes) +
                                        (r >> 1) * S::kRowPair + (r & 1) * D + lane * E;
#pragma unroll
                    for (int i = 0; i < E; i += 2) {
                        const float2 y = *reinterpret_cast<const float2 *>(from + i);
                        v[i] = fmaf(y.x, f, v[i]), v[i + 1] = fmaf(y.y, f, v[i + 1]);
                    }
                }
            }
            if (d1 > d0) {
                float qv[E];
                kvq_row<E>(a.q, a.type, (n * a.Hq + hq) * D + lane * E, qv);
                bool bad = false;
#pragma unroll
                for (int i = 0; i < E; ++i) bad = bad || !(fabsf(qv[i]) < kKvqLargestQ);
                bad = __any_sync(0xffffffffu, bad);
                const uint64_t *mask = a.mask + n * a.words;
                const int64_t base = (static_cast<int64_t>(s.h) * a.drafts + s.req.n0) * D + lane * E;
                for (int w0 = d0; w0 < d1; w0 += 64) {  // (kKvqTile is a multiple of 64)
                    uint64_t seen = mask[w0 >> 6];
                    if (d1 - w0 < 64) seen &= (1ull << (d1 - w0)) - 1;
                    while (seen) {
                        constexpr int kBatch = 4;
                        int64_t at[kBatch];
                        float kv[kBatch][E], vv[kBatch][E], sc[kBatch];
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            at[k] = seen ? base + static_cast<int64_t>(w0 + __ffsll(static_cast<long long>(seen)) - 1) * D : -1;
                            seen &= seen - 1;
                            if (at[k] < 0) continue;
                            kvq_row<E>(a.Kd, a.type, at[k], kv[k]);
                            kvq_row<E>(a.Vd, a.type, at[k], vv[k]);
                        }
                        float top = M;
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            sc[k] = 0.0f;
                            if (at[k] >= 0)
#pragma unroll
                                for (int i = 0; i < E; ++i) sc[k] = fmaf(qv[i], kv[k][i], sc[k]);
                        }
#pragma unroll
                        for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
                            for (int k = 0; k < kBatch; ++k) sc[k] += __shfl_xor_sync(0xffffffffu, sc[k], d);
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            sc[k] = at[k] < 0 ? -INFINITY : bad ? __int_as_float(0x7fc00000) : sc[k] * p.scale2;
                            top = fmaxf(top, sc[k]);
                        }
                        const float ref = top == -INFINITY ? 0.0f : top, f = exp2f(M - ref);
                        M = top;
                        L *= f;
#pragma unroll
                        for (int i = 0; i < E; ++i) v[i] *= f;
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            if (at[k] < 0) continue;
                            const float w = exp2f(sc[k] - ref);
                            L += w;
#pragma unroll
                            for (int i = 0; i < E; ++i) v[i] = fmaf(w, vv[k][i], v[i]);
                        }
                    }
                }
            }
            if (whole) {
                if (a.y_type == ABG_SB_F32) {
                    attn_finish<float, D>(a, n, hq, v, L);
                } else if (a.y_type == ABG_SB_BF16) {
                    attn_finish<__nv_bfloat16, D>(a, n, hq, v, L);
                } else {
                    attn_finish<__half, D>(a, n, hq, v, L);
                }
            } else {
                float *po = p.part_o + (slot * kRT + r) * D + lane * E;
#pragma unroll
                for (int i = 0; i < E; ++i) po[i] = v[i];
                if (lane == 0) p.part_ml[slot * kRT + r] = make_float2(M, L);
            }
        }
        if (tid == 0) line.leave_entry(p, s, blockIdx.x, left);
        __syncthreads();  // the rings and the rows' factors are free
    }
    if (tid == 0) line.end_entries(p, blockIdx.x, left);
}

template <typename S>
cudaError_t kvq_go(KvqAttnArgs x, void *ws, bool early, bool pdl, cudaStream_t stream) {
    const int C = std::min(S::kBlocks * sm_count(), kMaxBlocks);
    static const cudaError_t attr =
        cudaFuncSetAttribute(kvq_attn_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (attr != cudaSuccess) return attr;
    const AttnLayout l = attn_layout(C, S::kRT, S::D);
    unsigned char *w = static_cast<unsigned char *>(ws);
    x.p.part_o = reinterpret_cast<float *>(w + l.o);
    x.p.part_ml = reinterpret_cast<float2 *>(w + l.ml);
    x.p.split = reinterpret_cast<AttnSplit *>(w + l.split);
    attn_entries(x.p, C, S::kRT);
    const cudaError_t e = launch_kernel(kvq_attn_kernel<S>, dim3(C), dim3(kKvqThreads), S::kSmem, stream, early, x);
    if (e != cudaSuccess) return e;
    switch (x.p.a.y_type) {
    case ABG_SB_F32: return launch_join<float, S::D, S::kRT, false>(x.p, C, pdl, stream);
    case ABG_SB_BF16: return launch_join<__nv_bfloat16, S::D, S::kRT, false>(x.p, C, pdl, stream);
    default: return launch_join<__half, S::D, S::kRT, false>(x.p, C, pdl, stream);
    }
}

// Rows of a tile: 8, 16 or (up to 128 columns) 32, as a request and head has them;
// more would not fit in the registers, and are tiles of their own, which read the
// cache again.
inline int kvq_row_tile(int64_t D, int64_t rows) { return rows <= 8 ? 8 : rows <= 16 || D == 256 ? 16 : 32; }

// f.template operator()<Shape>() for the cache's format and a call's rows; f16 and
// f32 queries take two terms
template <int D, int kBits, typename F>
auto kvq_by_rows(int group, int rt, bool split, F f) {
    auto nt = [&](auto g, auto sp) {
        constexpr int G = decltype(g)::value;
        constexpr bool kSp = decltype(sp)::value;
        if constexpr (D < 256) {
            if (rt == 32) return f.template operator()<KvqShape<D, kBits, G, 4, kSp>>();
        }
        return rt == 8 ? f.template operator()<KvqShape<D, kBits, G, 1, kSp>>()
                       : f.template operator()<KvqShape<D, kBits, G, 2, kSp>>();
    };
    auto sp = [&](auto g) { return split ? nt(g, std::true_type{}) : nt(g, std::false_type{}); };
    return group == 32 ? sp(std::integral_constant<int, 32>{}) : sp(std::integral_constant<int, 64>{});
}

struct KvqGo {
    const KvqAttnArgs &x;
    void *ws;
    bool early, pdl;
    cudaStream_t stream;
    template <typename S>
    cudaError_t operator()() const {
        return kvq_go<S>(x, ws, early, pdl, stream);
    }
};
struct KvqBytes {
    template <typename S>
    size_t operator()() const {
        return attn_layout(std::min(S::kBlocks * sm_count(), kMaxBlocks), S::kRT, S::D).total;
    }
};

// one translation unit a width and number of bits
template <int D, int kBits>
cudaError_t kvq_attn_launch(const KvqAttnArgs &x, int group, int rt, bool split, void *ws, bool early, bool pdl,
                            cudaStream_t stream);

}  // namespace abg
