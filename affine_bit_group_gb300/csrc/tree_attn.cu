// tree_attn: attention of drafted tokens over a paged cache and one another
// (formulas in include/abg.h, the work split in tree_attn.cuh).  This file holds
// the f32 kernel, whose products are f32 on the CUDA cores: the tensor cores
// would round its operands.
#include "abg_kernels.cuh"
#include "tree_attn.cuh"
#include "tree_attn16.cuh"

#include <algorithm>
#include <cmath>

namespace abg {

namespace {

constexpr int kThreads = 256;

// Rows of a unit: 4, 8 or 16 where a request has no more, else 32 (8 rows on 32
// requests of 4100 tokens, 256 columns: in units of 16 121 us, of 8 96, now 91).  A block
// with a tile and 32 rows of 256 columns takes half of an SM's shared memory:
// two blocks an SM fill the gaps between each other's barriers (8 drafts over
// 60000 tokens, 128 columns: 88 us against 98 with one block of 64 rows and 64
// tokens, before the scores were a warp's own; now 72).
constexpr int kOneRows = 4, kEightRows = 8, kFewRows = 16, kManyRows = 32;

__device__ __forceinline__ void cp16(void *dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(real ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int kRT>
struct Smem {
    // Tokens a tile: what two blocks an SM have room for, since a tile costs three
    // barriers whatever its size (64 columns, 32 rows: 32 tokens 46.6 us, 64 40.5,
    // 128 in one stage 43.2; 16 rows: 32 tokens 101, 64 86, 128 79; 128 columns, 4
    // rows: two stages of 32 171 us, one of 64 138, now 134.5, 6.0 TB/s).
    static constexpr int kKT = D == 256 ? 32 : D == 128 || kRT == kManyRows ? 64 : 128;
    static constexpr int kLd = D + 4;                        // rows of Q and K start in different banks
    static constexpr int kPLd = kRT + 4;
    static constexpr bool kRowWarps = kRT >= kFewRows;       // a warp's scores are of rows of its own
    static constexpr int kParts = kRowWarps ? 1 : kThreads / kKT;  // else: column parts of the scores
    // K and V tiles in use and on their way
    static constexpr int kStages = D == 64 && kRT == kManyRows ? 2 : 1;
    alignas(16) float q[kRT][kLd];
    alignas(16) float k[kStages][kKT][kLd];
    alignas(16) float v[kStages][kKT][D];
    alignas(16) float p[kKT][kPLd];                    // weights, token-major
    float part[kParts][kRowWarps ? 1 : kRT][kKT + 1];  // partial scores
    alignas(16) float corr[kRT];                       // read in pairs
    int64_t off[4][kKT];                               // row offsets of tiles in turn, in elements (-1: none)
    float m[kRT], l[kRT];
    AttnScan scan;
    uint32_t bad[ABG_MAX_SPAN / 32];                   // drafts whose V holds an infinity or a NaN
};

template <int D, int kKT>
__device__ __forceinline__ void load_tile(float *dst, int ld, const float *src, const int64_t *off, int tokens) {
    constexpr int kEach = kKT * (D / 4) / kThreads, kRows = kThreads / (D / 4);  // rows of a round
    const int r0 = threadIdx.x / (D / 4), c = 4 * (threadIdx.x % (D / 4));
    if (tokens == kKT) {  // rounds side by side: their places are read before any is needed
        int64_t o[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) o[u] = off[r0 + u * kRows];
#pragma unroll
        for (int u = 0; u < kEach; ++u)
            cp16(dst + (r0 + u * kRows) * ld + c, src + max(o[u], int64_t(0)) + c, o[u] >= 0);
    } else {
        for (int r = r0; r < tokens; r += kRows)
            cp16(dst + r * ld + c, src + max(off[r], int64_t(0)) + c, off[r] >= 0);
    }
}

// Tile t of a stretch: tokens key0 .. key0+tokens-1 of the cache or of the drafts.
struct Tile {
    bool cache;
    int key0, tokens;
};
template <int kKT>
__device__ __forceinline__ Tile tile_at(const AttnSeg &s, int t) {
    Tile x;
    x.cache = t < s.ctiles;
    x.key0 = (x.cache ? t : t - s.ctiles) * kKT;
    x.tokens = min(kKT, (x.cache ? s.req.len : s.req.T) - x.key0);
    return x;
}

// Page of the tile's token i (0 for drafts), and, given it, where the token's row
// lies (in elements of its tensor; -1: nowhere).  In two steps, so that the
// table's latency passes during another tile's work.
__device__ __forceinline__ int32_t page_of(const abg_tree_attn_args &a, const AttnSeg &s, const Tile &x, int i) {
    if (!x.cache || i >= x.tokens) return 0;
    return a.table[static_cast<int64_t>(s.b) * a.width + static_cast<uint32_t>(x.key0 + i) / static_cast<uint32_t>(a.page)];
}
template <int D>
__device__ __forceinline__ int64_t row_offset(const abg_tree_attn_args &a, const AttnSeg &s, const Tile &x, int i,
                                              int32_t id) {
    if (i >= x.tokens) return -1;
    if (!x.cache) return (s.h * a.drafts + s.req.n0 + x.key0 + i) * static_cast<int64_t>(D);
    if (id < 0 || id >= a.pages) return -1;
    const uint32_t in_page = static_cast<uint32_t>(x.key0 + i) % static_cast<uint32_t>(a.page);
    return ((static_cast<int64_t>(id) * a.Hkv + s.h) * a.page + in_page) * D;
}

// Sums over the D/8 lanes of a token group of 16 values, rows x tokens.  Half of
// the values go to the other half of the lanes in each step; what is left of
// them is the row and the token at index 16/R * row + token = the lane's place.
// The rows' steps come first, of the most values: a lane's rows start from its
// own (x[i] is row i ^ its row), so that these steps select nothing.
template <int D, int R>
__device__ __forceinline__ void scatter_sums(float (&x)[16], int lane) {
#pragma unroll
    for (int half = 8, d = D / 16; half >= (D == 64 ? 2 : 1); half /= 2, d /= 2) {
        const bool up = half < 16 / R && lane & d;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = up ? x[i + half] : x[i], send = up ? x[i] : x[i + half];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, d);
        }
    }
}

// One part of the work line.  Scores of 16 or 32 rows: a warp has 2 or 4 rows of
// its own, a lane eight of their columns in registers; K goes past them, a token
// to every D/8 lanes, and the lanes' sums meet by shuffles, 16 values at a time,
// which leaves each lane the scores of one row, so that the softmax needs no
// shared memory and no barrier before it.  (Rows of Q read from shared memory
// again for every token took 70 us where this took 65, now 62.9: 8 drafts of 8 heads on
// four ragged f32 requests of 4100 tokens, 256 columns.)  Up to 8 rows: a thread
// holds a part of the columns of one token for all rows, and the parts meet in
// shared memory (8 rows on 32 requests of 4100 tokens: 91 us, 4.4 TB/s; with a
// row a warp 15 more).
// Weighted sums: a thread holds four columns of kRPO rows, two rows to a packed
// pair, over every kKS-th token.  Multiply-adds bound it above about 16 rows (half
// a multiply-add a byte and row, against 11 a byte that an SM can do): they keep
// their units busy 40-50% of the time and half of the instructions are others, at
// 16 warps an SM, which is as many as the registers hold.  Below, latency and the
// cache's bytes.
template <int D, int kRT>
__global__ void __launch_bounds__(kThreads, 2) attn_kernel(const __grid_constant__ AttnArgs p) {
    using S = Smem<D, kRT>;
    extern __shared__ __align__(16) unsigned char raw[];
    S &sm = *reinterpret_cast<S *>(raw);
    const abg_tree_attn_args &a = p.a;
    constexpr int kParts = S::kParts, kKT = S::kKT;
    constexpr bool kRowWarps = S::kRowWarps;
    constexpr int kLanes = kThreads / kRT < 32 ? kThreads / kRT : 32;  // of a row's softmax
    constexpr int kEach = kKT / kLanes;                                // a lane's tokens of it
    constexpr int kRW = kRowWarps ? kRT / (kThreads / 32) : 1;         // rows of a warp
    constexpr int kTS = 16 / kRW;                                      // tokens of a lane at a time
    constexpr int kRPO = kRT < 8 ? kRT : 8;                            // rows of a thread's sums
    constexpr int kQuads = D / 4, kRG = kRT / kRPO, kKS = kThreads / (kQuads * kRG);
    constexpr int E = D / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // softmax: a thread's row, and 0 in the first of the threads that share it
    // (kRowWarps: from the lane's place that scatter_sums goes by)
    const int place16 = D == 256 ? lane >> 1 : D == 128 ? lane & 15 : 2 * (lane & 7);
    constexpr int kRowBits = (kRW - 1) * kTS * D / 128;  // lanes of one row differ elsewhere
    const int row = kRowWarps ? kRW * warp + place16 / kTS : tid / kLanes;
    const int col = kRowWarps ? lane & ~kRowBits : tid % kLanes;
    const int quad = tid % kQuads, rg = tid / kQuads % kRG, ks = tid / (kQuads * kRG);
    grid_dep_wait();
    grid_dep_launch();
    AttnLine<kRT, kKT> line;
    line.template init<kThreads>(p, blockIdx.x, gridDim.x, sm.scan);
    bool left = false;
    AttnSeg s;
    while (line.next(p, s)) {
        // whole warps (they shuffle) have softmax rows or not
        const bool rows_here = kRowWarps ? kRW * warp < s.rows : (32 * warp) / kLanes < s.rows && row < kRT;
        auto source = [&](const Tile &x, bool value) {
            return static_cast<const float *>(x.cache ? (value ? a.Vc : a.Kc) : (value ? a.Vd : a.Kd));
        };
        constexpr int kStages = S::kStages;
        const int n = s.t1 - s.t0;
        __syncthreads();  // the last stretch's shared memory is done with
        int32_t id = 0;   // page of the token that this thread looks up next
        if (tid < kKT) {
#pragma unroll
            for (int u = 0; u < kStages; ++u)
                if (u < n) {
                    const Tile x = tile_at<kKT>(s, s.t0 + u);
                    sm.off[u][tid] = row_offset<D>(a, s, x, tid, page_of(a, s, x, tid));
                }
            if (kStages < n) id = page_of(a, s, tile_at<kKT>(s, s.t0 + kStages), tid);
        }
        for (int i = tid; i < kRT * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4)), q = s.r0 + r;
            const bool in = r < s.rows;
            cp16(&sm.q[r][c],
                 static_cast<const float *>(a.q) +
                     (in ? ((static_cast<int64_t>(s.req.n0) + q / p.G) * a.Hq + s.h * p.G + q % p.G) * D + c : 0),
                 in);
        }
        if (tid < ABG_MAX_SPAN / 32) sm.bad[tid] = 0;
        __syncthreads();
        auto bring = [&](int u, bool value) {  // tile u of the stretch (Q goes with the first); a group each
            if (u < n) {
                const Tile x = tile_at<kKT>(s, s.t0 + u);
                if (value) {
                    load_tile<D, kKT>(&sm.v[u % kStages][0][0], D, source(x, true), sm.off[u & 3], x.tokens);
                } else {
                    load_tile<D, kKT>(&sm.k[u % kStages][0][0], S::kLd, source(x, false), sm.off[u & 3], x.tokens);
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int u = 0; u < kStages; ++u) bring(u, false), bring(u, true);
        float m = -INFINITY, l = 0.0f;
        float4 q[kRW][2];       // columns 4l .. 4l+3 and D/2 further on of a warp's rows
        float2 o[kRPO / 2][4];  // rows 2i and 2i+1, a column
#pragma unroll
        for (int i = 0; i < kRPO / 2; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = make_float2(0.0f, 0.0f);
        for (int u = 0; u < n; ++u) {
            const Tile now = tile_at<kKT>(s, s.t0 + u);
            const int st = u % kStages;
            // the places of tile u + kStages, and the pages of the one after it
            if (tid < kKT && u + kStages < n) {
                sm.off[(u + kStages) & 3][tid] = row_offset<D>(a, s, tile_at<kKT>(s, s.t0 + u + kStages), tid, id);
                if (u + kStages + 1 < n) id = page_of(a, s, tile_at<kKT>(s, s.t0 + u + kStages + 1), tid);
            }
            cp_wait<2 * kStages - 1>();
            __syncthreads();
            // scores
            if constexpr (!kRowWarps) {
                const int key = tid % kKT, part = tid / kKT;
                if (key < now.tokens) {
                    float2 acc[kRT];
#pragma unroll
                    for (int r = 0; r < kRT; ++r) acc[r] = make_float2(0.0f, 0.0f);
#pragma unroll 4
                    for (int c = part * (D / kParts); c < (part + 1) * (D / kParts); c += 4) {
                        const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[st][key][c]);
#pragma unroll
                        for (int r = 0; r < kRT; ++r) {
                            const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[r][c]);
                            acc[r] = fma2(make_float2(qv.x, qv.y), make_float2(kv.x, kv.y), acc[r]);
                            acc[r] = fma2(make_float2(qv.z, qv.w), make_float2(kv.z, kv.w), acc[r]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < kRT; ++r) sm.part[part][r][key] = acc[r].x + acc[r].y;
                }
                __syncthreads();
                bring(u + kStages, false);
            }
            // softmax statistics and weights
            if (rows_here) {
                const uint64_t *seen = nullptr;
                if (!now.cache && row < s.rows)
                    seen = a.mask + (static_cast<int64_t>(s.req.n0) + (s.r0 + row) / p.G) * a.words;
                float sc[kEach], top = m;
                int at[kEach];
                if constexpr (kRowWarps) {
                    constexpr int kGroups = 256 / D;  // of lanes, a token each
                    const int g = lane / (D / 8), c = 4 * (lane % (D / 8));
                    if (u == 0)
#pragma unroll
                        for (int i = 0; i < kRW; ++i) {
                            q[i][0] = *reinterpret_cast<const float4 *>(&sm.q[kRW * warp + (i ^ place16 / kTS)][c]);
                            q[i][1] = *reinterpret_cast<const float4 *>(&sm.q[kRW * warp + (i ^ place16 / kTS)][D / 2 + c]);
                        }
                    constexpr int kLeft = D == 64 ? 2 : 1;
                    constexpr int kPasses = kKT / (kTS * kGroups);
                    float half = 0.0f;
#pragma unroll
                    for (int t = 0; t < kPasses; ++t) {
                        float v[16];
#pragma unroll
                        for (int j = 0; j < kTS; ++j) {
                            const float *k = &sm.k[st][(t * kGroups + g) * kTS + j][c];
                            const float4 k0 = *reinterpret_cast<const float4 *>(k);
                            const float4 k1 = *reinterpret_cast<const float4 *>(k + D / 2);
#pragma unroll
                            for (int i = 0; i < kRW; ++i) {
                                float2 x = mul2(make_float2(q[i][0].x, q[i][0].y), make_float2(k0.x, k0.y));
                                x = fma2(make_float2(q[i][0].z, q[i][0].w), make_float2(k0.z, k0.w), x);
                                x = fma2(make_float2(q[i][1].x, q[i][1].y), make_float2(k1.x, k1.y), x);
                                x = fma2(make_float2(q[i][1].z, q[i][1].w), make_float2(k1.z, k1.w), x);
                                v[i * kTS + j] = x.x + x.y;
                            }
                        }
                        scatter_sums<D, kRW>(v, lane);
                        if constexpr (D == 256) {  // two passes' sums meet in lane pairs
                            if (t % 2 == 0) {
                                half = v[0];
                            } else {
                                const bool up = lane & 1;
                                const float send = up ? half : v[0], keep = up ? v[0] : half;
                                sc[t / 2] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < kLeft; ++e) sc[t * kLeft + e] = v[e];
                        }
                    }
                    const int j0 = place16 % kTS;
#pragma unroll
                    for (int n = 0; n < kEach; ++n)
                        at[n] = D == 256   ? (2 * n + (lane & 1)) * kTS + j0
                                : D == 128 ? (n * kGroups + g) * kTS + j0
                                           : (n / 2 * kGroups + g) * kTS + j0 + n % 2;
                } else {
#pragma unroll
                    for (int j = 0; j < kEach; ++j) {
                        at[j] = col + kLanes * j;
                        float x[kParts];
#pragma unroll
                        for (int h = 0; h < kParts; ++h) x[h] = sm.part[h][row][at[j]];
#pragma unroll
                        for (int w = kParts / 2; w >= 1; w /= 2)
#pragma unroll
                            for (int h = 0; h < w; ++h) x[h] = x[2 * h] + x[2 * h + 1];
                        sc[j] = x[0];
                    }
                }
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    const bool in =
                        at[j] < now.tokens && (now.cache || (seen && attn_sees(seen, now.key0 + at[j])));
                    sc[j] = in ? sc[j] * p.scale2 : -INFINITY;
                    top = fmaxf(top, sc[j]);
                }
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1)
                    if (kRowWarps ? !(d & kRowBits) : d < kLanes) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float ref = top == -INFINITY ? 0.0f : top;
                const float corr = exp2f(m - ref);
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    const float e = exp2f(sc[j] - ref);
                    sum += e;
                    sm.p[at[j]][row] = e;
                }
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1)
                    if (kRowWarps ? !(d & kRowBits) : d < kLanes) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                l = l * corr + sum;
                m = top;
                if (col == 0) sm.corr[row] = corr;
            }
            cp_wait<2 * kStages - (kRowWarps ? 2 : 1)>();
            __syncthreads();
            if constexpr (kRowWarps) bring(u + kStages, false);
            if (!now.cache) {
                // an infinity or a NaN in a draft's V must not reach the rows
                // that do not see it (0 * NaN): taken out here, and added at the
                // end to the rows that do
                for (int i = tid; i < now.tokens * D; i += kThreads) {
                    float &v = sm.v[st][i / D][i % D];
                    if (!(fabsf(v) < INFINITY)) {
                        v = 0.0f;
                        const int k = now.key0 + i / D;
                        atomicOr(&sm.bad[k >> 5], 1u << (k & 31));
                    }
                }
                __syncthreads();
            }
            // weighted sums
#pragma unroll
            for (int i = 0; i < kRPO / 2; ++i) {
                const float2 f = *reinterpret_cast<const float2 *>(&sm.corr[rg * kRPO + 2 * i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] = mul2(o[i][e], f);
            }
            auto take = [&](int k) {
                const float4 v = *reinterpret_cast<const float4 *>(&sm.v[st][k][4 * quad]);
                const float2 vv[4] = {make_float2(v.x, v.x), make_float2(v.y, v.y), make_float2(v.z, v.z),
                                      make_float2(v.w, v.w)};
#pragma unroll
                for (int i = 0; i < kRPO / 2; i += 2) {
                    const float4 w = *reinterpret_cast<const float4 *>(&sm.p[k][rg * kRPO + 2 * i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[i][e] = fma2(make_float2(w.x, w.y), vv[e], o[i][e]);
                        o[i + 1][e] = fma2(make_float2(w.z, w.w), vv[e], o[i + 1][e]);
                    }
                }
            };
            if (rg * kRPO >= s.rows) {  // no rows
            } else if (now.tokens == kKT) {  // written out (a loop of unknown length: 78.9 us where this takes 71.0)
#pragma unroll 32
                for (int k = 0; k < kKT; k += kKS) take(ks + k);
            } else {
#pragma unroll 1
                for (int k = ks; k < now.tokens; k += kKS) take(k);
            }
            __syncthreads();
            bring(u + kStages, true);
        }
        cp_wait<0>();
        // the token groups' sums, halving the groups each time, through the
        // memory of the K and V tiles; then [kRT][D] there
        float *os = &sm.k[0][0][0];
        static_assert(sizeof(float) * kRT * D * (kKS > 1 ? kKS / 2 : 1) <= sizeof sm.k + sizeof sm.v, "groups' sums");
        auto place = [&](int g, int i, int h) {
            return reinterpret_cast<float4 *>(os + (g * kRT + rg * kRPO + 2 * i + h) * D + 4 * quad);
        };
#pragma unroll
        for (int g = kKS / 2; g >= 1; g /= 2) {
            if (ks >= g && ks < 2 * g)
#pragma unroll
                for (int i = 0; i < kRPO / 2; ++i) {
                    *place(ks - g, i, 0) = make_float4(o[i][0].x, o[i][1].x, o[i][2].x, o[i][3].x);
                    *place(ks - g, i, 1) = make_float4(o[i][0].y, o[i][1].y, o[i][2].y, o[i][3].y);
                }
            __syncthreads();
            if (ks < g)
#pragma unroll
                for (int i = 0; i < kRPO / 2; ++i) {
                    const float4 x = *place(ks, i, 0), y = *place(ks, i, 1);
                    o[i][0] = add2(o[i][0], make_float2(x.x, y.x)), o[i][1] = add2(o[i][1], make_float2(x.y, y.y));
                    o[i][2] = add2(o[i][2], make_float2(x.z, y.z)), o[i][3] = add2(o[i][3], make_float2(x.w, y.w));
                }
            __syncthreads();
        }
        if (ks == 0)
#pragma unroll
            for (int i = 0; i < kRPO / 2; ++i) {
                *place(0, i, 0) = make_float4(o[i][0].x, o[i][1].x, o[i][2].x, o[i][3].x);
                *place(0, i, 1) = make_float4(o[i][0].y, o[i][1].y, o[i][2].y, o[i][3].y);
            }
        if (col == 0 && rows_here) sm.m[row] = m, sm.l[row] = l;
        __syncthreads();
        const bool whole = s.t0 == 0 && s.t1 == s.tiles;
        const int64_t slot = static_cast<int64_t>(2) * blockIdx.x + (s.t0 == 0);
        for (int r = warp; r < s.rows; r += kThreads / 32) {
            float v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = os[r * D + lane * E + i];
            const int64_t n = static_cast<int64_t>(s.req.n0) + (s.r0 + r) / p.G;
            for (int w = 0; w < (s.req.T + 31) / 32; ++w)
                for (uint32_t b = sm.bad[w]; b; b &= b - 1) {
                    const int k = 32 * w + __ffs(static_cast<int>(b)) - 1;
                    if (!attn_sees(a.mask + n * a.words, k)) continue;
                    const float *row = static_cast<const float *>(a.Vd) + (s.h * a.drafts + s.req.n0 + k) * static_cast<int64_t>(D);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float x = row[lane * E + i];
                        if (!(fabsf(x) < INFINITY)) v[i] += x;
                    }
                }
            if (whole) {
                attn_finish<float, D>(a, n, s.h * p.G + (s.r0 + r) % p.G, v, sm.l[r]);
            } else {
                float *po = p.part_o + (slot * kRT + r) * D + lane * E;
#pragma unroll
                for (int i = 0; i < E; ++i) po[i] = v[i];
                if (lane == 0) p.part_ml[slot * kRT + r] = make_float2(sm.m[r], sm.l[r]);
            }
        }
        if (tid == 0) line.leave_entry(p, s, blockIdx.x, left);
    }
    if (tid == 0) line.end_entries(p, blockIdx.x, left);
}

int row_tile(int64_t G, int64_t max_span) {
    const int64_t rows = G * max_span;
    return rows <= kOneRows     ? kOneRows
           : rows <= kEightRows ? kEightRows
           : rows <= kFewRows   ? kFewRows
                                : kManyRows;
}

template <int D, int kRT>
int grid_of() {
    static const int blocks = [] {
        int per = 0;
        if (cudaFuncSetAttribute(attn_kernel<D, kRT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 sizeof(Smem<D, kRT>)) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, attn_kernel<D, kRT>, kThreads,
                                                          sizeof(Smem<D, kRT>)) != cudaSuccess)
            per = 1;
        return std::min(std::max(1, per) * sm_count(), kMaxBlocks);
    }();
    return blocks;
}

template <int D, int kRT>
cudaError_t go(AttnArgs p, void *ws, bool early, bool pdl, cudaStream_t stream) {
    const int C = grid_of<D, kRT>();
    const AttnLayout l = attn_layout(C, kRT, D);
    unsigned char *w = static_cast<unsigned char *>(ws);
    p.part_o = reinterpret_cast<float *>(w + l.o);
    p.part_ml = reinterpret_cast<float2 *>(w + l.ml);
    p.split = reinterpret_cast<AttnSplit *>(w + l.split);
    attn_entries(p, C, kRT);
    const cudaError_t e =
        launch_kernel(attn_kernel<D, kRT>, dim3(C), dim3(kThreads), sizeof(Smem<D, kRT>), stream, early, p);
    if (e != cudaSuccess) return e;
    return launch_join<float, D, kRT, false>(p, C, pdl, stream);
}

// f.template operator()<D, kRT>() for the call's width and rows
template <int D, typename F>
auto by_rows(int rt, F f) {
    return rt == kOneRows     ? f.template operator()<D, kOneRows>()
           : rt == kEightRows ? f.template operator()<D, kEightRows>()
           : rt == kFewRows   ? f.template operator()<D, kFewRows>()
                              : f.template operator()<D, kManyRows>();
}
template <typename F>
auto by_shape(int64_t D, int rt, F f) {
    return D == 64 ? by_rows<64>(rt, f) : D == 128 ? by_rows<128>(rt, f) : by_rows<256>(rt, f);
}
struct Bytes {
    template <int D, int kRT>
    size_t operator()() const {
        return attn_layout(grid_of<D, kRT>(), kRT, D).total;
    }
};
struct Go {
    const AttnArgs &p;
    void *ws;
    bool early, pdl;
    cudaStream_t stream;
    template <int D, int kRT>
    cudaError_t operator()() const {
        return go<D, kRT>(p, ws, early, pdl, stream);
    }
};

}  // namespace

size_t tree_attn_bytes(int Hq, int Hkv, int D, int max_span, int type) {
    return type == ABG_SB_F32 ? by_shape(D, row_tile(Hq / Hkv, max_span), Bytes{}) : tree_attn16_bytes(D);
}

cudaError_t launch_tree_attn(const abg_tree_attn_args &a, void *ws, bool pdl, int withhold, cudaStream_t stream) {
    AttnArgs p{};
    p.a = a;
    p.G = static_cast<int>(a.Hq / a.Hkv);
    p.scale2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.D)));
    const bool early = pdl && !capturing(stream);
    return a.type == ABG_SB_F32 ? by_shape(a.D, row_tile(p.G, a.max_span), Go{p, ws, early, pdl, stream})
                                : launch_tree_attn16(p, ws, early, pdl, withhold, stream);
}

}  // namespace abg
