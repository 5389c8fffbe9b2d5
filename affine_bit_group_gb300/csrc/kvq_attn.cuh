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
// Warps.  Every warp goes through blocks of 16 or 32 tokens of its own (every eighth of
// the stretch), with a ring in shared memory that it fills by cp.async and its own
// reference and sums: no barrier until the stretch's end, where the warps' sums meet in
// shared memory.  The drafts are multiplied in f32, a few lanes a row, while the first
// blocks are on their way, and what a stretch needs besides is asked for before its
// copies, behind which it would wait.
//
// What bounds it.  64 requests of up to 16000 tokens, 16 heads over 4 of 128 columns, 4
// bits, take 102 us for 441 MB (4.3 TB/s): copies alone take about 70, the rest without
// copies about 75, with 600 instructions a warp for 32 tokens, half of them for taking the
// codes apart, and no one of them that shortens the call by more than 6 us when it is left
// out; launches, the joining and two beginnings and ends a block are 15 of it.  In 8 bits 48
// requests of 9001 tokens of 256 columns take 69 us (354 MB, 5.1 TB/s), one f16 token over
// 131071 28 us (75 MB), one over 2000 13 to 15 us, the latency of two launches.
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

constexpr int kKvqJoin = 8;    // pieces of a row that a warp has on their way when it joins
constexpr int kKvqTile = 128;  // tokens of the work line's tiles
// Rows of q from here on give NaN: their scores could pass f32's range.
constexpr float kKvqLargestQ = 1.2676506e30f;  // 2^100
// A score (in base 2) whose product with the row's factor rounds by up to 2^-2.
constexpr float kKvqFar = 4194304.0f;  // 2^22

template <int D_, int kBits_, int kGroup_, int kNT_, bool kSplit_>
struct KvqShape {
    static constexpr int D = D_, kBits = kBits_, kGroup = kGroup_;
    static constexpr int kNT = kNT_;                      // query rows, by 8
    static constexpr int kTerms = kSplit_ ? 2 : 1;        // f16 terms of q and of P
    // two terms: codes as normal numbers around 0 (K's c - kMiddle, V's c - z), else as
    // subnormal ones
    static constexpr bool kNormal = kSplit_;
    static constexpr float kMiddle = kNormal ? (kBits == 4 ? 8.0f : 128.0f) : 0.0f;
    static constexpr float kUnit = kNormal ? 1.0f : 16777216.0f;             // 1 / the operand's value of a code 1
    static constexpr float kUpper = !kNormal && kBits == 4 ? 16.0f : 1.0f;   // an upper nibble's over a lower's
    static constexpr int kRT = 8 * kNT;
    static constexpr int kRB = D * kBits / 8;             // bytes of a row's codes
    static constexpr int kG = D / kGroup, kFB = 4 * kG;   // groups of a row, bytes of its factors
    static constexpr int kTB = kRB <= 128 ? 32 : 16;       // tokens of a block
    static constexpr int kMT = kTB / 16;
    static constexpr int kSteps = D / 16;                 // products of 16 columns
    static constexpr int kWords = kGroup * kBits / 128;   // words of a group in a lane
    // Blocks an SM.  The sums take kNT * D / 4 registers of a lane; up to 32, two blocks of
    // 128 registers that go through 16 tokens at a time stand against one of up to 255 that
    // goes through 32.  64 requests of 8000 tokens, us of two and of one, bf16 / f32 queries:
    //   64 columns,  8 rows, 4 bits, groups of 64    78 and 102 / 108 and 129
    //                                groups of 32    86 and 105 / 123 and 141
    //                        8 bits, groups of 64    98 and 122 / 119 and 145
    //                                groups of 32   101 and 121 / 132 and 151
    //   64 columns, 16 rows, 4 bits, groups of 64   137 and 141 / 185 and 168
    //                                groups of 32   178 and 151 / 230 and 196
    //                        8 bits, groups of 64   148 and 162 / 200 and 188
    //                                groups of 32   212 and 171 / 247 and 209
    //   128 columns, 8 rows, 4 bits, groups of 64    74 and  75 / 106 and 107
    //                                groups of 32    86 and  86 / 122 and 122
    // The 16-row shapes of 64 columns spill 84 to 344 bytes a thread in two blocks, and only
    // bf16 in groups of 64 gains by them all the same; those of 128 columns spill 60 to 140.
    // Two blocks that go through 32 tokens at a time spill more (128 columns, bf16, groups of
    // 64: 103 us for 101; of 32: 86 for 75).  With 64 registers of sums, two blocks would spill
    // all the more, and 12 warps of 168 registers do no more.
    static constexpr int kBlocks = kNT * D / 4 <= 32 && kRB <= 64 ? 2 : 1;
    static constexpr int kMP = kBlocks == 2 ? 1 : kMT;    // 16-token tiles of a block side by side
    static constexpr int kWarps = 8, kThreads = 32 * kWarps;
    static constexpr int kL = kThreads / kRT, kE = D / kL;  // lanes of a row for drafts and result, columns of a lane
    static constexpr int kStageBytes = kTB * 2 * (kRB + kFB);
    static constexpr int kQBytes = kSteps * kTerms * kNT * 32 * 8;
    // a warp's factors of a block: f32 pairs of K and of V; f16 -(1024 + z) of V
    static constexpr int kFacBytes = kTB * kG * (16 + (kNormal ? 2 : 0));
    // (its place holds q's rows in f32 before)
    static constexpr int kFacAll = std::max(kWarps * kFacBytes, kRT * (D + 4) * 4);
    static constexpr int kPark = kBlocks == 2 ? kRT * (D + 2) * 4 : 0;  // the drafts' part of the rows' sums
    static constexpr int kFixed = kQBytes + 4 * kRT * (kG + 1 + 2 * kWarps) + kFacAll + (kPark + 15) / 16 * 16;
    static constexpr int kRoom = (kBlocks == 2 ? 113 : 226) * 1024 - kFixed - 1024;
    static constexpr int kStages = std::min(6, kRoom / (kWarps * kStageBytes));
    static constexpr int kRowPair = 2 * D + 2;            // floats of two rows of a warp's sums
    static constexpr int kWarpBytes = std::max(kStages * kStageBytes, kRT / 2 * kRowPair * 4 + 8) / 16 * 16;
    static_assert(kStages >= 2 && kWarpBytes * kWarps <= kRoom, "the ring fits");
    static constexpr int kSmem = kFixed + kWarps * kWarpBytes;
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
// d = a b
__device__ __forceinline__ void kvq_mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y), "f"(0.0f));
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
// conflicts left, but for 8 bits in groups of 64 of a 64-column row, 24 for 16).  An XOR of
// t's lowest three bits, so that the place of a sum of tokens is the XOR of theirs.
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

// E columns from `at` on of y, of the sums v and the weight l (attn_finish of E columns
// a lane); all lanes call it, `mine` says which write.
template <int E>
__device__ __forceinline__ void kvq_finish(const abg_tree_attn_args &a, int64_t at, float (&v)[E], float l, bool mine) {
    float sum = 0.0f;
    if (mine) {
        if (a.gate) {
            float g[E];
            load_e<float, E>(a.gate + at, g);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = (l == 0.0f ? 0.0f : v[i] / l) * (1.0f / (1.0f + expf(-g[i])));
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = l == 0.0f ? 0.0f : v[i] / l;
        }
        if (a.y_type == ABG_SB_F32) {
            store_e<float, E>(static_cast<float *>(a.y) + at, v);
        } else if (a.y_type == ABG_SB_BF16) {
            store_e<__nv_bfloat16, E>(static_cast<__nv_bfloat16 *>(a.y) + at, v);
        } else {
            store_e<__half, E>(static_cast<__half *>(a.y) + at, v);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) sum += v[i];
    }
    if (a.ysum) {
#pragma unroll
        for (int d = 1; d < 64 / E; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (mine && at % 64 == 0) a.ysum[at / 64] = sum;
    }
}

template <typename S>
__global__ void __launch_bounds__(S::kThreads, S::kBlocks) kvq_attn_kernel(const __grid_constant__ KvqAttnArgs x) {
    constexpr int D = S::D, kNT = S::kNT, kRT = S::kRT, kRB = S::kRB, kFB = S::kFB, kG = S::kG, kTB = S::kTB;
    constexpr int kMT = S::kMT, kMP = S::kMP, kTerms = S::kTerms, kStages = S::kStages, kGroup = S::kGroup, kBits = S::kBits;
    constexpr int E = D / 32, kTiles = D / 16, kWarps = S::kWarps, kThreads = S::kThreads;
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ AttnScan scan;
    // (in shared memory while the blocks go by, so that no register holds them)
    using Line = AttnLine<kRT, kKvqTile>;
    __shared__ Line s_line, s_next;           // and the next stretch's
    __shared__ AttnSeg s_seg[2];              // this stretch and the next
    __shared__ bool s_more;
    __shared__ const int32_t *s_table;        // the request's row
    const AttnArgs &p = x.p;
    const abg_tree_attn_args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j = lane >> 2, quad = lane & 3;
    uint2 *s_q = reinterpret_cast<uint2 *>(raw);                            // [step][term][row tile][lane]
    float *s_qs = reinterpret_cast<float *>(raw + S::kQBytes);              // [kG][kRT] group sums of q
    float *s_f = s_qs + kG * kRT;                                           // [kRT] factor of a row's scores
    float *s_m = s_f + kRT, *s_l = s_m + kWarps * kRT;                   // [warp][kRT]
    // the block's factors in f32, two groups of a token side by side: [kG / 2][kTB][2] pairs
    float *s_qf = s_l + kWarps * kRT;                                       // [kRT][D + 4] (before the factors)
    float *s_park = reinterpret_cast<float *>(reinterpret_cast<unsigned char *>(s_qf) + S::kFacAll);  // [kRT][D], [kRT][2]
    float2 *k_fac = reinterpret_cast<float2 *>(s_qf) + warp * (S::kFacBytes / 8);
    float2 *v_fac = k_fac + kTB * kG;
    __half *zero = reinterpret_cast<__half *>(v_fac + kTB * kG);            // [kG][kTB], by pairs of tokens
    constexpr int kPair = kG > 1 ? 2 : 1;
    unsigned char *ring = raw + (S::kFixed + warp * S::kWarpBytes);
    const uint32_t ring_at = smem_u32(ring);
    static_assert(S::kFixed % 16 == 0, "the ring's alignment");
    grid_dep_wait();
    grid_dep_launch();
    // row r of a unit's q: which of q's rows of D values
    auto q_row = [&](const AttnSeg &s, int r) {
        const int q = s.r0 + r, draft = q / p.G;
        return (static_cast<int64_t>(s.req.n0) + draft) * a.Hq + s.h * p.G + (q - draft * p.G);
    };
    bool left = false;
    {
        Line line;
        line.template init<kThreads>(p, blockIdx.x, gridDim.x, scan);
        if (tid == 0) {
            s_more = line.next(p, s_seg[0]);
            s_line = line;
        }
        __syncthreads();
    }
    for (int turn = 0;; turn ^= 1) {
        if (!s_more) break;
        AttnSeg s = s_seg[turn];
        if (tid == 0) s_table = a.table + static_cast<int64_t>(s.b) * a.width;
        __syncthreads();
        const int key0 = min(s.t0, s.ctiles) * kKvqTile;
        const int key1 = min(s.req.len, min(s.t1, s.ctiles) * kKvqTile);    // cached tokens of the stretch
        // -- what is asked for first: q, a row a warp, and the masks of the drafts' part,
        // kL lanes a row; later they would wait behind the copies --
        constexpr int kRows = kRT / kWarps;
        float q[kRows][E];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int r = k * kWarps + warp;
#pragma unroll
            for (int i = 0; i < E; ++i) q[k][i] = 0.0f;
            if (r < s.rows) kvq_row<E>(a.q, a.type, q_row(s, r) * D + lane * E, q[k]);
        }
        constexpr int kL = S::kL, kE = S::kE;
        const int r = warp * (32 / kL) + lane / kL, ln = lane % kL;
        const bool mine = r < s.rows;
        const int d0 = (max(s.t0, s.ctiles) - s.ctiles) * kKvqTile, d1 = min(s.req.T, (s.t1 - s.ctiles) * kKvqTile);
        auto word = [&](int w0) -> uint64_t {  // drafts w0 .. w0 + 63 that the row sees (kKvqTile is a multiple of 64)
            if (!mine || w0 >= d1) return 0;
            const int64_t n = static_cast<int64_t>(s.req.n0) + (s.r0 + r) / p.G;
            const uint64_t seen = a.mask[n * a.words + (w0 >> 6)];
            return d1 - w0 < 64 ? seen & ((1ull << (d1 - w0)) - 1) : seen;
        };
        uint64_t seen = word(d0);
        // -- copies --
        auto page_at = [&](int t) {
            return x.page_mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(t), x.page_mul) >> x.page_shift) : t;
        };
        int t_next = key0 + warp * kTB + lane;  // this lane's token of the block that is brought next
        auto page_of = [&](int t) { return lane < kTB && t < key1 ? s_table[page_at(t)] : -1; };
        int32_t id, ids[kStages];               // and its page
#pragma unroll
        for (int i = 0; i < kStages; ++i) ids[i] = page_of(t_next + i * kWarps * kTB);
        // the drafts that the row sees, some at a time: their rows on their way, then their
        // weights and sums
        constexpr int kBatch = kE > 4 ? 2 : 4;
        const int64_t base = (static_cast<int64_t>(s.h) * a.drafts + s.req.n0) * D + ln * kE;
        int64_t d_at[kBatch];
        float d_k[kBatch][kE], d_v[kBatch][kE];
        auto ask = [&](int w0) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                d_at[k] = seen ? base + static_cast<int64_t>(w0 + __ffsll(static_cast<long long>(seen)) - 1) * D : -1;
                seen &= seen - 1;
                if (d_at[k] < 0) continue;
                kvq_row<kE>(a.Kd, a.type, d_at[k], d_k[k]);
                kvq_row<kE>(a.Vd, a.type, d_at[k], d_v[k]);
            }
        };
        if (d1 > d0) ask(d0);
        auto bring = [&](int stage) {           // that block; a group of copies
            if (t_next - lane < key1) {
                const int page = static_cast<int>(a.page);
                const bool there = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.pages);
                // (a cache has fewer than 2^32 rows)
                const uint32_t row = there ? (static_cast<uint32_t>(id) * static_cast<uint32_t>(a.Hkv) + s_seg[turn].h) * page +
                                                 (t_next - page_at(t_next) * page)
                                           : 0;
                t_next += kWarps * kTB;
                const uint32_t at = ring_at + stage * S::kStageBytes;
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
        for (int i = 0; i < kStages - 1; ++i) {
            id = ids[i];
            bring(i);
        }
        id = ids[kStages - 1];
        // -- q: a row a warp for its scale and sums, then the products' operands --
        {
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int qr = k * kWarps + warp;
                float top = 0.0f, sum = 0.0f;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    top = fabsf(q[k][i]) < INFINITY ? fmaxf(top, fabsf(q[k][i])) : INFINITY;
                    sum += q[k][i];
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
                if (lane == 1) s_l[qr] = 1.0f / up;  // (until the drafts are done)
                if (lane == 0) s_f[qr] = bad ? __int_as_float(0x7fc00000) : p.scale2 * S::kUnit / up;
                if (lane % (kGroup / E) == 0) s_qs[lane / (kGroup / E) * kRT + qr] = sum * up * (1.0f / S::kUnit);
#pragma unroll
                for (int i = 0; i < E; ++i) s_qf[qr * (D + 4) + lane * E + i] = q[k][i] * up;
            }
            __syncthreads();
#pragma unroll 2
            for (int i = tid; i < S::kSteps * kNT * 32; i += kThreads) {
                const int ln = i & 31, nt = i / 32 % kNT, step = i / (32 * kNT);
                constexpr int kPerWord = kBits == 4 ? 2 : 1;  // steps of a word
                const int w = step / kPerWord, g = w / S::kWords, wi = w % S::kWords;
                const int col = g * kGroup + ((ln & 3) * S::kWords + wi) * (32 / kBits) + (kBits == 4 ? 2 * (step % 2) : 0);
                // the pairs' columns: 0 and 4, 1 and 5 of 4 bits (the second a nibble up:
                // 2^4), 0 and 2, 1 and 3 of 8
                constexpr int kNext = kBits == 4 ? 4 : 2;
                const float *from = s_qf + (nt * 8 + (ln >> 2)) * (D + 4) + col;
                const float v0 = from[0], v1 = from[kNext], v2 = from[1] * (1.0f / S::kUpper), v3 = from[kNext + 1] * (1.0f / S::kUpper);
                uint2 *to = s_q + ((step * kTerms) * kNT + nt) * 32 + ln;
                const uint2 hi = make_uint2(kvq_half2(v0, v1), kvq_half2(v2, v3));
                *to = hi;
                if constexpr (kTerms == 2) {
                    const float2 h0 = kvq_float2(hi.x), h1 = kvq_float2(hi.y);
                    to[kNT * 32] = make_uint2(kvq_half2(v0 - h0.x, v1 - h0.y), kvq_half2(v2 - h1.x, v3 - h1.y));
                }
            }
        }
        // -- the drafts --
        float d_m = -INFINITY, d_l = 0.0f, d_o[kE];
#pragma unroll
        for (int i = 0; i < kE; ++i) d_o[i] = 0.0f;
        if (d1 > d0) {
            float qv[kE];
#pragma unroll
            for (int i = 0; i < kE; ++i) qv[i] = s_qf[r * (D + 4) + ln * kE + i] * s_l[r];  // (as it was: K has f32's range)
            const float f = s_f[r] == s_f[r] ? p.scale2 : __int_as_float(0x7fc00000);
            for (int w0 = d0;;) {
                float sc[kBatch], top = d_m;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    sc[k] = 0.0f;
                    if (d_at[k] >= 0)
#pragma unroll
                        for (int i = 0; i < kE; ++i) sc[k] = fmaf(qv[i], d_k[k][i], sc[k]);
                }
#pragma unroll
                for (int d = kL / 2; d >= 1; d >>= 1)
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) sc[k] += __shfl_xor_sync(0xffffffffu, sc[k], d);
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    sc[k] = d_at[k] < 0 ? -INFINITY : sc[k] * f;
                    top = fmaxf(top, sc[k]);
                }
                const float ref = top == -INFINITY ? 0.0f : top, corr = exp2f(d_m - ref);
                d_m = top;
                d_l *= corr;
#pragma unroll
                for (int i = 0; i < kE; ++i) d_o[i] *= corr;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    if (d_at[k] < 0) continue;
                    const float w = exp2f(sc[k] - ref);
                    d_l += w;
#pragma unroll
                    for (int i = 0; i < kE; ++i) d_o[i] = fmaf(w, d_v[k][i], d_o[i]);
                }
                while (!__any_sync(0xffffffffu, seen != 0) && w0 < d1) seen = word(w0 += 64);
                if (w0 >= d1) break;
                ask(w0);
            }
        }
        if constexpr (S::kPark > 0) {
#pragma unroll
            for (int i = 0; i < kE; ++i) s_park[r * D + ln * kE + i] = d_o[i];
            if (ln == 0) s_park[kRT * D + 2 * r] = d_m, s_park[kRT * D + 2 * r + 1] = d_l;
        }
        __syncthreads();
        // the next stretch, whose numbers come while the blocks go by
        if (tid == kThreads - 32) {
            Line line = s_line;
            s_more = line.next(p, s_seg[turn ^ 1]);
            s_next = line;
        }
        // -- the warp's blocks --
        float o[kTiles][kNT][4];             // columns (8 or 4 a lane of a group, two a tile) x rows 2 quad, + 1
        float l[kNT][2], m[kNT][2], bias[kG][kNT][2];
        // up brings the largest scale of V so far to 2^13 .. 2^14, down its products' results
        // back; one of these f16 bits is twice as large or more (at first: any that is not 0)
        float up = pow2i(37), down = pow2i(-37) * S::kUnit;
        uint32_t larger = 1;
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
        int stage = 0;
        for (int t0 = key0 + warp * kTB; t0 < key1; t0 += kWarps * kTB) {
            kvq_wait<kStages - 2>();
            __syncwarp();  // every lane's copies have come, and the last block's place is free
            bring(stage == 0 ? kStages - 1 : stage - 1);
            id = page_of(t_next);
            const unsigned char *K = ring + stage * S::kStageBytes, *V = K + kTB * kRB, *Kf = V + kTB * kRB,
                                *Vf = Kf + kTB * kFB;
            // the factors, a token a lane; V's scales times a power of two that brings the
            // largest so far to 2^13 .. 2^14
            {
                uint32_t kf[kG], vf[kG], big = 0;
                if (lane < kTB) {
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        kf[g] = *reinterpret_cast<const uint32_t *>(Kf + lane * kFB + 4 * g);
                        vf[g] = *reinterpret_cast<const uint32_t *>(Vf + lane * kFB + 4 * g);
                        const uint32_t v = vf[g] & 0x7fffu;
                        big = max(big, v < 0x7c00u ? v : 0u);
                    }
                }
                if (__any_sync(0xffffffffu, big >= larger)) {
                    // (as a f32, where f16's subnormal numbers have exponents of their own)
                    const float top = kvq_float2(__reduce_max_sync(0xffffffffu, big)).x;
                    const int ev = static_cast<int>(__float_as_uint(top) >> 23) - 127;
                    up = pow2i(13 - ev);
                    down = pow2i(ev - 13) * S::kUnit;
                    larger = __half_as_ushort(__float2half_rn(pow2i(ev + 1)));
                }
                if (lane < kTB) {
                    float2 kk[kG], vv[kG];
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        kk[g] = kvq_float2(kf[g]);
                        vv[g] = kvq_float2(vf[g]);
                        if constexpr (S::kNormal) {
                            kk[g].y = fmaf(S::kMiddle, kk[g].x, kk[g].y);
                            // (any z is right; no scale, or a NaN: one of the ends)
                            const float z =
                                fminf(fmaxf(rintf(__fdividef(-vv[g].y, vv[g].x)), 0.0f), kBits == 4 ? 15.0f : 255.0f);
                            vv[g].y = fmaf(vv[g].x, z, vv[g].y);
                            zero[g * kTB + (lane & ~7) + 2 * (lane & 3) + (lane >> 2 & 1)] = __float2half_rn(-1024.0f - z);
                        }
                        vv[g].x *= up;
                    }
#pragma unroll
                    for (int g = 0; g < kG; g += kPair) {
                        float2 *const kt = k_fac + g * kTB + lane * kPair, *const vt = v_fac + g * kTB + lane * kPair;
                        if constexpr (kPair == 2) {
                            *reinterpret_cast<float4 *>(kt) = make_float4(kk[g].x, kk[g].y, kk[g + 1].x, kk[g + 1].y);
                            *reinterpret_cast<float4 *>(vt) = make_float4(vv[g].x, vv[g].y, vv[g + 1].x, vv[g + 1].y);
                        } else {
                            *kt = kk[g];
                            *vt = vv[g];
                        }
                    }
                }
                __syncwarp();
            }
            // scale and bias of token t, groups g (even) and g + 1
            auto factors = [&](const float2 *fac, int t, int g, float2 (&f)[2]) {
                const float2 *from = fac + g * kTB + t * kPair;
                if constexpr (kPair == 2) {
                    const float4 v = *reinterpret_cast<const float4 *>(from);
                    f[0] = make_float2(v.x, v.y), f[1] = make_float2(v.z, v.w);
                } else {
                    f[0] = *from;
                }
            };
            // scores
            float sc[kMT][kNT][4];
            float2 f2[kMP][2][2];  // of tokens tok and tok + 8, of two groups
#pragma unroll
            for (int m0 = 0; m0 < kMT; m0 += kMP) {
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                if (g % 2 == 0)
#pragma unroll
                    for (int mt = m0; mt < m0 + kMP; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) factors(k_fac, 16 * mt + 8 * h + tok, g, f2[mt - m0][h]);
                uint32_t w[kMP][2][S::kWords];
#pragma unroll
                for (int mt = m0; mt < m0 + kMP; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int off = g * (kGroup * kBits / 8) + quad * (4 * S::kWords);
                        const unsigned char *from =
                            K + (16 * mt + 8 * h + tok) * kRB + (((off >> 4) ^ kvq_swizzle<S>(tok)) << 4) + (off & 15);
                        if constexpr (S::kWords == 1) {
                            w[mt - m0][h][0] = *reinterpret_cast<const uint32_t *>(from);
                        } else if constexpr (S::kWords == 2) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(from);
                            w[mt - m0][h][0] = v.x, w[mt - m0][h][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4 *>(from);
                            w[mt - m0][h][0] = v.x, w[mt - m0][h][1] = v.y, w[mt - m0][h][2] = v.z, w[mt - m0][h][3] = v.w;
                        }
                    }
                float acc[kMP][kNT][4];
                constexpr int kPerWord = kBits == 4 ? 2 : 1;
#pragma unroll
                for (int wi = 0; wi < S::kWords; ++wi)
#pragma unroll
                    for (int hh = 0; hh < kPerWord; ++hh) {
                        const int step = (g * S::kWords + wi) * kPerWord + hh;
                        uint32_t e[kMP][4];
#pragma unroll
                        for (int mt = m0; mt < m0 + kMP; ++mt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t v = w[mt - m0][h][wi] >> (8 * hh);
                                const __half2 from = __float2half2_rn(-1024.0f - S::kMiddle);
                                e[mt - m0][h] = kvq_operand<S, false>(v, from);
                                e[mt - m0][2 + h] = kvq_operand<S, true>(v, from);
                            }
#pragma unroll
                        for (int term = 0; term < kTerms; ++term)
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt) {
                                const uint2 b = s_q[((step * kTerms + term) * kNT + nt) * 32 + lane];
#pragma unroll
                                for (int mt = m0; mt < m0 + kMP; ++mt) {
                                    if (wi == 0 && hh == 0 && term == 0) {
                                        kvq_mma0(acc[mt - m0][nt], e[mt - m0][0], e[mt - m0][1], e[mt - m0][2], e[mt - m0][3], b);
                                    } else {
                                        kvq_mma(acc[mt - m0][nt], e[mt - m0][0], e[mt - m0][1], e[mt - m0][2], e[mt - m0][3], b);
                                    }
                                }
                            }
                    }
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    const float2 qs = *reinterpret_cast<const float2 *>(s_qs + g * kRT + nt * 8 + 2 * quad);
#pragma unroll
                    for (int mt = m0; mt < m0 + kMP; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = f2[mt - m0][e >> 1][g % 2];
                            const float qe = e & 1 ? qs.y : qs.x;
                            sc[mt][nt][e] = fmaf(acc[mt - m0][nt][e], f.x, g == 0 ? f.y * qe : fmaf(f.y, qe, sc[mt][nt][e]));
                        }
                }
            }
            }
            // maxima and weights: sc and m are in units of 1/s_f, so that the largest score is m
            // itself and not m as a product rounds it (which from 2^23 on could be off by a
            // weight that passes f16's range, or by all of the weights)
            const int here = key1 - t0;  // tokens of the block that are there
            if (here < kTB) {
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (16 * mt + 8 * (e >> 1) + tok >= here) sc[mt][nt][e] = -INFINITY;
            }
            // the rows' reference m goes up, and their sums down, where a score lies more
            // than 1.5 above it: weights are below 2^1.5, which f16 has room for
            bool above = false;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const float2 f = *reinterpret_cast<const float2 *>(s_f + nt * 8 + 2 * quad);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(sc[0][nt][e], sc[0][nt][2 + e]);
                    if constexpr (kMT == 2) top = fmaxf(top, fmaxf(sc[kMT - 1][nt][e], sc[kMT - 1][nt][2 + e]));
                    above = above || (top - m[nt][e]) * (e ? f.y : f.x) > 1.5f;
                }
            }
            if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    const float2 f = *reinterpret_cast<const float2 *>(s_f + nt * 8 + 2 * quad);
                    float corr[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(sc[0][nt][e], sc[0][nt][2 + e]);
                        if constexpr (kMT == 2) top = fmaxf(top, fmaxf(sc[kMT - 1][nt][e], sc[kMT - 1][nt][2 + e]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        top = fmaxf(m[nt][e], top);
                        corr[e] = kvq_exp2((m[nt][e] - (top == -INFINITY ? 0.0f : top)) * (e ? f.y : f.x));
                        m[nt][e] = top;
                        l[nt][e] *= corr[e];
#pragma unroll
                        for (int g = 0; g < kG; ++g) bias[g][nt][e] *= corr[e];
                    }
#pragma unroll
                    for (int k = 0; k < kTiles; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[k][nt][e] *= corr[e & 1];
                }
            }
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const float2 f = *reinterpret_cast<const float2 *>(s_f + nt * 8 + 2 * quad);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float &v = sc[mt][nt][2 * h + e];
                            v = kvq_exp2((v - ref) * (e ? f.y : f.x));
                            l[nt][e] += v;
                        }
                }
            }
            // weighted sums
#pragma unroll
            for (int m0 = 0; m0 < kMT; m0 += kMP) {
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                if (g % 2 == 0)
#pragma unroll
                    for (int mt = m0; mt < m0 + kMP; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) factors(v_fac, 16 * mt + 8 * h + tok, g, f2[mt - m0][h]);
                constexpr int kCols = kGroup / 8, kColWords = kCols * kBits > 32 ? kCols * kBits / 32 : 1;
                uint2 b[kMP][kTerms][kNT];
                uint32_t u[kMP][4][kColWords];
                __half2 z[kMP][2];
#pragma unroll
                for (int mt = m0; mt < m0 + kMP; ++mt) {
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
                        const float *w = sc[mt][nt];
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = f2[mt - m0][e >> 1][g % 2];
                            v[e] = w[e] * f.x;
                            bias[g][nt][e & 1] = fmaf(w[e], f.y, bias[g][nt][e & 1]);
                        }
                        const uint32_t h0 = kvq_half2(v[0], v[1]), h1 = kvq_half2(v[2], v[3]);
                        b[mt - m0][0][nt] = make_uint2(kvq_transpose(h0), kvq_transpose(h1));
                        if constexpr (kTerms == 2) {
                            const float2 r0 = kvq_float2(h0), r1 = kvq_float2(h1);
                            b[mt - m0][1][nt] = make_uint2(kvq_transpose(kvq_half2(v[0] - r0.x, v[1] - r0.y)),
                                                      kvq_transpose(kvq_half2(v[2] - r1.x, v[3] - r1.y)));
                        }
                    }
                    // the lane's columns of the group, of tokens quad, + 4, + 8, + 12, and where their codes
                    // are counted from
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // (the group's and the token's part of the chunk's place are the same for all lanes)
                        const int off = kCols * kBits / 8 * j & ~3, same = g * (kGroup * kBits / 128) ^ kvq_swizzle<S>(4 * (k & 1));
                        const unsigned char *from = V + (16 * mt + 4 * k) * kRB + quad * kRB + (off & 15) +
                                                    (((off >> 4) ^ kvq_swizzle<S>(quad) ^ same) << 4);
                        if constexpr (kColWords == 2) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(from);
                            u[mt - m0][k][0] = v.x, u[mt - m0][k][1] = v.y;
                        } else {
                            u[mt - m0][k][0] = *reinterpret_cast<const uint32_t *>(from);
                        }
                    }
                    if constexpr (S::kNormal) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            z[mt - m0][k] = *reinterpret_cast<const __half2 *>(zero + g * kTB + 16 * mt + 8 * k + 2 * quad);
                    }
                }
#pragma unroll
                for (int i = 0; i < kGroup / 16; ++i) {  // columns 2 i and 2 i + 1 of the lane's
                    float part[kNT][4];                  // of the block
#pragma unroll
                    for (int mt = m0; mt < m0 + kMP; ++mt) {
                        uint32_t e[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {  // tokens quad and + 4, then + 8 and + 12
                            // 4 bits: four columns of both tokens; 8: two
                            const int word = kBits == 4 ? 0 : i / 2;
                            const bool upper = kBits == 8 ? i % 2 : kGroup == 32 ? j & 1 : i >= 2;
                            uint32_t v = __byte_perm(u[mt - m0][2 * k][word], u[mt - m0][2 * k + 1][word], upper ? 0x7632u : 0x5410u);
                            if (kBits == 4) v >>= 8 * (i % 2);
                            e[2 * k] = kvq_operand<S, false>(v, z[mt - m0][k]), e[2 * k + 1] = kvq_operand<S, true>(v, z[mt - m0][k]);
                        }
#pragma unroll
                        for (int term = 0; term < kTerms; ++term)
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt) {
                                if (mt == m0 && term == 0) {
                                    kvq_mma0(part[nt], e[0], e[1], e[2], e[3], b[mt - m0][term][nt]);
                                } else {
                                    kvq_mma(part[nt], e[0], e[1], e[2], e[3], b[mt - m0][term][nt]);
                                }
                            }
                    }
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float &sum = o[g * (kGroup / 16) + i][nt][e];
                            sum = fmaf(part[nt][e], e < 2 ? down : down * (1.0f / S::kUpper), sum);
                        }
                }
            }
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        kvq_wait<0>();
        __syncwarp();
        // -- the warp's sums to shared memory, in its ring --
        const bool cached = key1 > key0;
        if (cached) {
            float *mine = reinterpret_cast<float *>(ring);
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
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float2 *>(mine + (nt * 4 + quad) * S::kRowPair + e * D + col) =
                            make_float2(o[i][nt][e] + bias[g][nt][e], o[i][nt][2 + e] + bias[g][nt][e]);
                }
            }
        }
        // -- kL lanes a row: the warps' sums, the drafts', the result --
        s = s_seg[turn];
        __syncthreads();
        float M, L, v[kE];
        if constexpr (S::kPark > 0) {
#pragma unroll
            for (int i = 0; i < kE; ++i) v[i] = s_park[r * D + ln * kE + i];
            M = s_park[kRT * D + 2 * r], L = s_park[kRT * D + 2 * r + 1];
        } else {
#pragma unroll
            for (int i = 0; i < kE; ++i) v[i] = d_o[i];
            M = d_m, L = d_l;
        }
        if (cached) {
            static_assert(kWarps == 8 && kL >= 8);
            const float mw = s_m[(ln & 7) * kRT + r], lw = s_l[(ln & 7) * kRT + r];
            float top = mw;
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float f = s_f[r];
            top = fmaxf(__fmul_rn(top, f), M);
            // what the rounding of a moderate maximum took is in the weights; that of a far one
            // is not, as it could be all of them
            const float over = fabsf(top) < kKvqFar ? fmaf(mw, f, -top) : __fsub_rn(__fmul_rn(mw, f), top);
            // (no maximum, but a weight: a NaN, which stays, as one that is far below does)
            const float fw = mw == -INFINITY ? 1.0f : exp2f(over);
            const float fd = M == -INFINITY ? 1.0f : exp2f(M - top);
            const bool none = L == 0.0f;
            M = top;
            L *= fd;
#pragma unroll
            for (int i = 0; i < kE; ++i) v[i] = none ? 0.0f : v[i] * fd;
#pragma unroll
            for (int u = 0; u < kWarps; ++u) {
                const float fu = __shfl_sync(0xffffffffu, fw, u, kL), lu = __shfl_sync(0xffffffffu, lw, u, kL);
                if (lu == 0.0f) continue;  // no token: nothing to add
                L = fmaf(lu, fu, L);
                const float *from = reinterpret_cast<const float *>(raw + S::kFixed + u * S::kWarpBytes) +
                                    (r >> 1) * S::kRowPair + (r & 1) * D + ln * kE;
#pragma unroll
                for (int i = 0; i < kE; i += 2) {
                    const float2 y = *reinterpret_cast<const float2 *>(from + i);
                    v[i] = fmaf(y.x, fu, v[i]), v[i + 1] = fmaf(y.y, fu, v[i + 1]);
                }
            }
        }
        if (s.t0 == 0 && s.t1 == s.tiles) {
            kvq_finish<kE>(a, q_row(s, mine ? r : 0) * D + ln * kE, v, L, mine);
        } else if (mine) {
            const int64_t slot = (static_cast<int64_t>(2) * blockIdx.x + (s.t0 == 0)) * kRT + r;
            float *po = p.part_o + slot * D + ln * kE;
#pragma unroll
            for (int i = 0; i < kE; i += 2) *reinterpret_cast<float2 *>(po + i) = make_float2(v[i], v[i + 1]);
            if (ln == 0) p.part_ml[slot] = make_float2(M, L);
        }
        if (tid == 0) {
            s_line.leave_entry(p, s, blockIdx.x, left);
            s_line = s_next;
        }
        __syncthreads();  // the rings and the rows' factors are free
    }
    if (tid == 0) s_line.end_entries(p, blockIdx.x, left);
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
    const cudaError_t e = launch_kernel(kvq_attn_kernel<S>, dim3(C), dim3(S::kThreads), S::kSmem, stream, early, x);
    if (e != cudaSuccess) return e;
    switch (x.p.a.y_type) {
    case ABG_SB_F32: return launch_join<float, S::D, S::kRT, false, kKvqJoin>(x.p, C, pdl, stream);
    case ABG_SB_BF16: return launch_join<__nv_bfloat16, S::D, S::kRT, false, kKvqJoin>(x.p, C, pdl, stream);
    default: return launch_join<__half, S::D, S::kRT, false, kKvqJoin>(x.p, C, pdl, stream);
    }
}

// Rows of a tile: 8, or 16 where a request and head has more and D is below 256, so that
// the sums take at most 64 registers of a lane; rows beyond are tiles of their own, which
// read the cache again.  (128 registers of sums, at 128 columns 32 rows a tile: eight f32
// drafts of four requests 44.7 us where two tiles take 26.7, four bf16 drafts of 32
// requests 117 and 76.6; at 256 columns 16 rows 118 and 96.6.  At 64 columns 32 rows fit,
// and take 50.6 us where 16 take 49.0.)
inline int kvq_row_tile(int64_t D, int64_t rows) { return rows <= 8 || D == 256 ? 8 : 16; }

// f.template operator()<Shape>() for the cache's format and a call's rows; f16 and
// f32 queries take two terms
template <int D, int kBits, typename F>
auto kvq_by_rows(int group, int rt, bool split, F f) {
    auto nt = [&](auto g, auto sp) {
        constexpr int G = decltype(g)::value;
        constexpr bool kSp = decltype(sp)::value;
        if constexpr (D < 256) {
            if (rt == 16) return f.template operator()<KvqShape<D, kBits, G, 2, kSp>>();
        }
        return f.template operator()<KvqShape<D, kBits, G, 1, kSp>>();
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
