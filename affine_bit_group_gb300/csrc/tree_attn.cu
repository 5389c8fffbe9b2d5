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

constexpr int kThreads = 512;
// The work line is cut at every 32 tokens, and a stretch is taken in tiles of
// up to 64: with the few tiles a block gets of f32 work (a tile of 64 rows is
// 8 us of an SM), the even split counts more than the tile.
constexpr int kKT = 32, kTile = 64;

// Rows of a unit: up to 4, 16 or 32 where a request has no more, else 64.
constexpr int kOneRows = 4, kFewRows = 16, kSomeRows = 32, kManyRows = 64;

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
    static constexpr int kLd = D + 4;                       // rows of Q and K start in different banks
    static constexpr int kPLd = kRT + 4;
    static constexpr int kWide = kRT > kFewRows;             // score tiles of 4 x 4 a thread
    static constexpr int kParts = kWide ? 8 * 16 / kRT : 8;  // column parts of the scores
    float q[kRT][kLd];
    float k[kTile][kLd];
    float v[kTile][D];
    float p[kTile][kPLd];                     // weights, token-major
    // partial scores: of all parts, or (wide) of the third part on
    float part[kWide ? kParts - 2 : kParts][kTile][kWide ? kPLd : kRT];
    float corr[kRT];
    int64_t off[2][kTile];                    // a tile's row offsets in elements (-1: none)
    float m[kRT], l[kRT];
    AttnScan scan;
    uint32_t bad[ABG_MAX_SPAN / 32];          // drafts whose V holds an infinity or a NaN
};

// Where token `key` of a stretch's request lies (in elements of its tensor), -1: nowhere.
template <int D>
__device__ __forceinline__ int64_t row_offset(const abg_tree_attn_args &a, const AttnSeg &s, bool cache, int key) {
    if (cache) {
        if (key >= s.req.len) return -1;
        const int j = static_cast<int>(key / static_cast<unsigned>(a.page));
        const int64_t id = a.table[static_cast<int64_t>(s.b) * a.width + j];
        if (id < 0 || id >= a.pages) return -1;
        return ((id * a.Hkv + s.h) * a.page + (key - static_cast<int64_t>(j) * a.page)) * D;
    }
    return key < s.req.T ? (s.h * a.drafts + s.req.n0 + key) * static_cast<int64_t>(D) : -1;
}

template <int D>
__device__ __forceinline__ void load_tile(float *dst, int ld, const float *src, const int64_t *off, int tokens) {
    for (int i = threadIdx.x; i < tokens * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        const int64_t o = off[r];
        cp16(dst + r * ld + c, src + max(o, int64_t(0)) + c, o >= 0);
    }
    cp_commit();
}

// A tile: tokens key0 .. key0+tokens-1 of the cache or of the drafts; `to` is
// the stretch's work after it.
struct Tile {
    bool cache;
    int key0, tokens, to;
};
__device__ __forceinline__ Tile tile_at(const AttnSeg &s, int t) {
    Tile x;
    x.cache = t < s.ctiles;
    x.to = min(t + kTile / kKT, x.cache ? min(s.ctiles, s.t1) : s.t1);
    x.key0 = (x.cache ? t : t - s.ctiles) * kKT;
    x.tokens = min((x.to - t) * kKT, (x.cache ? s.req.len : s.req.T) - x.key0);
    return x;
}

// One part of the work line.  Scores: up to 16 rows, a thread holds an eighth of
// the columns of one token for all rows, and the eighths meet in shared memory;
// 32 or 64 rows, a quarter or half of the columns of four rows by four tokens.  Then thread (ty,
// tx) = (tid / 16, tid % 16) has the scores of kRPS rows and tokens tx + 16 j.  Sums: a thread
// holds four columns of kRPO rows, two rows to a packed pair, over every
// kKS-th token.  f32 arithmetic is what bounds it above about 16 rows (0.5
// multiply-adds a byte and row against 11 a byte that an SM can do); below,
// latency and the cache's bytes.
template <int D, int kRT>
__global__ void __launch_bounds__(kThreads) attn_kernel(const __grid_constant__ AttnArgs p) {
    using S = Smem<D, kRT>;
    extern __shared__ __align__(16) unsigned char raw[];
    S &sm = *reinterpret_cast<S *>(raw);
    const abg_tree_attn_args &a = p.a;
    constexpr int kRPS = S::kWide ? 4 : 1;           // rows of a softmax thread
    constexpr int kTY = S::kWide ? kRT / 4 : 32;     // thread rows of a score tile
    constexpr int kParts = S::kParts;
    constexpr int kRPO = kRT < 8 ? kRT : 8;        // rows of a thread's sums
    constexpr int kQuads = D / 4, kRG = kRT / kRPO, kKS = kThreads / (kQuads * kRG);
    constexpr int E = D / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tx = tid % 16, ty = (tid % (16 * kTY)) / 16;
    const int quad = tid % kQuads, rg = tid / kQuads % kRG, ks = tid / (kQuads * kRG);
    grid_dep_wait();
    grid_dep_launch();
    AttnLine<kRT, kKT> line;
    line.template init<kThreads>(p, blockIdx.x, gridDim.x, sm.scan);
    bool left = false;
    AttnSeg s;
    while (line.next(p, s)) {
        const bool rows_here = 2 * kRPS * warp < s.rows;  // the warp has softmax rows (whole warps: they shuffle)
        const int part = tid / (S::kWide ? 16 * kTY : kTile);  // of the columns
        auto source = [&](const Tile &x, bool value) {
            return static_cast<const float *>(x.cache ? (value ? a.Vc : a.Kc) : (value ? a.Vd : a.Kd));
        };
        Tile now = tile_at(s, s.t0);
        __syncthreads();  // the last stretch's shared memory is done with
        if (tid < kTile) sm.off[0][tid] = row_offset<D>(a, s, now.cache, now.key0 + tid);
        for (int i = tid; i < kRT * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4)), row = s.r0 + r;
            const bool in = r < s.rows;
            cp16(&sm.q[r][c],
                 static_cast<const float *>(a.q) +
                     (in ? ((static_cast<int64_t>(s.req.n0) + row / p.G) * a.Hq + s.h * p.G + row % p.G) * D + c : 0),
                 in);
        }
        if (tid < ABG_MAX_SPAN / 32) sm.bad[tid] = 0;
        __syncthreads();
        load_tile<D>(&sm.k[0][0], S::kLd, source(now, false), sm.off[0], now.tokens);  // with Q: one group
        load_tile<D>(&sm.v[0][0], D, source(now, true), sm.off[0], now.tokens);
        float m[kRPS], l[kRPS];
        float2 o[kRPO / 2][4];  // rows 2i and 2i+1, a column
#pragma unroll
        for (int i = 0; i < kRPS; ++i) m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < kRPO / 2; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = make_float2(0.0f, 0.0f);
        for (int buf = 0, t = s.t0; t < s.t1; buf ^= 1) {
            const bool more = now.to < s.t1;
            const Tile next = more ? tile_at(s, now.to) : now;
            if (more && tid < kTile) sm.off[buf ^ 1][tid] = row_offset<D>(a, s, next.cache, next.key0 + tid);
            cp_wait<1>();
            __syncthreads();
            // scores
            float sc[kRPS][4];
            if constexpr (!S::kWide) {
                const int key = tid % kTile;
                if (key < now.tokens) {
                    float2 acc[kRT];
#pragma unroll
                    for (int r = 0; r < kRT; ++r) acc[r] = make_float2(0.0f, 0.0f);
#pragma unroll 2
                    for (int c = part * (D / 8); c < (part + 1) * (D / 8); c += 4) {
                        const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[key][c]);
#pragma unroll
                        for (int r = 0; r < kRT; ++r) {
                            const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[r][c]);
                            acc[r] = fma2(make_float2(qv.x, qv.y), make_float2(kv.x, kv.y), acc[r]);
                            acc[r] = fma2(make_float2(qv.z, qv.w), make_float2(kv.z, kv.w), acc[r]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < kRT; r += 4)
                        *reinterpret_cast<float4 *>(&sm.part[part][key][r]) =
                            make_float4(acc[r].x + acc[r].y, acc[r + 1].x + acc[r + 1].y, acc[r + 2].x + acc[r + 2].y,
                                        acc[r + 3].x + acc[r + 3].y);
                }
                __syncthreads();
                if (rows_here)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x[8];
#pragma unroll
                        for (int h = 0; h < 8; ++h) x[h] = sm.part[h][tx + 16 * j][ty];
                        sc[0][j] = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
                    }
            } else {
                const bool work = 8 * (warp % (kTY / 2)) < s.rows;  // the warp's eight rows
                auto scores = [&](auto keys) {
                    constexpr int kKeys = decltype(keys)::value;
                    float2 acc[kRPS][kKeys];
#pragma unroll
                    for (int i = 0; i < kRPS; ++i)
#pragma unroll
                        for (int j = 0; j < kKeys; ++j) acc[i][j] = make_float2(0.0f, 0.0f);
#pragma unroll 2
                    for (int c = part * (D / kParts); c < (part + 1) * (D / kParts); c += 4) {
                        float4 kv[kKeys];
#pragma unroll
                        for (int j = 0; j < kKeys; ++j)
                            kv[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][c]);
#pragma unroll
                        for (int i = 0; i < kRPS; ++i) {
                            const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[ty * kRPS + i][c]);
#pragma unroll
                            for (int j = 0; j < kKeys; ++j) {
                                acc[i][j] = fma2(make_float2(qv.x, qv.y), make_float2(kv[j].x, kv[j].y), acc[i][j]);
                                acc[i][j] = fma2(make_float2(qv.z, qv.w), make_float2(kv[j].z, kv[j].w), acc[i][j]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kRPS; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sc[i][j] = j < kKeys ? acc[i][j < kKeys ? j : 0].x + acc[i][j < kKeys ? j : 0].y : 0.0f;
                };
                if (work) {
                    if (now.tokens > 32) {
                        scores(std::integral_constant<int, 4>{});
                    } else {
                        scores(std::integral_constant<int, 2>{});
                    }
                    // the second part's go through the weights' memory
                    if (part)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float *to = &sm.p[tx + 16 * j][ty * 4];
                            if (kParts > 2 && part > 1) to = &sm.part[part - 2][tx + 16 * j][ty * 4];
                            *reinterpret_cast<float4 *>(to) = make_float4(sc[0][j], sc[1][j], sc[2][j], sc[3][j]);
                        }
                }
                __syncthreads();
                if (rows_here)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int h = 1; h < kParts; ++h) {
                            const float *from = h == 1 ? &sm.p[tx + 16 * j][ty * 4]
                                                       : &sm.part[h > 1 ? h - 2 : 0][tx + 16 * j][ty * 4];
                            const float4 x = *reinterpret_cast<const float4 *>(from);
                            sc[0][j] += x.x, sc[1][j] += x.y, sc[2][j] += x.z, sc[3][j] += x.w;
                        }
            }
            if (more) {
                load_tile<D>(&sm.k[0][0], S::kLd, source(next, false), sm.off[buf ^ 1], next.tokens);
            } else {
                cp_commit();
            }
            // softmax statistics and weights
            if (rows_here) {
#pragma unroll
                for (int i = 0; i < kRPS; ++i) {
                    const int r = ty * kRPS + i;
                    const uint64_t *seen = nullptr;
                    if (!now.cache && r < s.rows)
                        seen = a.mask + (static_cast<int64_t>(s.req.n0) + (s.r0 + r) / p.G) * a.words;
                    float top = m[i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = tx + 16 * j;
                        const bool in = k < now.tokens && (now.cache || (seen && attn_sees(seen, now.key0 + k)));
                        sc[i][j] = in ? sc[i][j] * p.scale2 : -INFINITY;
                        top = fmaxf(top, sc[i][j]);
                    }
#pragma unroll
                    for (int d = 8; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    const float corr = exp2f(m[i] - ref);
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sc[i][j] = exp2f(sc[i][j] - ref);
                        sum += sc[i][j];
                    }
#pragma unroll
                    for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    l[i] = l[i] * corr + sum;
                    m[i] = top;
                    if (tx == 0) sm.corr[r] = corr;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float *to = &sm.p[tx + 16 * j][ty * kRPS];
                    if constexpr (kRPS == 4) {
                        *reinterpret_cast<float4 *>(to) = make_float4(sc[0][j], sc[1][j], sc[2][j], sc[3][j]);
                    } else {
                        *to = sc[0][j];
                    }
                }
            }
            cp_wait<1>();
            __syncthreads();
            if (!now.cache) {
                // an infinity or a NaN in a draft's V must not reach the rows
                // that do not see it (0 * NaN): taken out here, and added at the
                // end to the rows that do
                for (int i = tid; i < now.tokens * D; i += kThreads) {
                    float &v = sm.v[i / D][i % D];
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
#pragma unroll 4
            for (int k = rg * kRPO < s.rows ? ks : now.tokens; k < now.tokens; k += kKS) {
                const float4 v = *reinterpret_cast<const float4 *>(&sm.v[k][4 * quad]);
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
            }
            __syncthreads();
            if (more) {
                load_tile<D>(&sm.v[0][0], D, source(next, true), sm.off[buf ^ 1], next.tokens);
            } else {
                cp_commit();
            }
            t = now.to;
            now = next;
        }
        cp_wait<0>();
        // the token groups' sums, halving the groups each time, through the
        // memory of the K and V tiles; then [kRT][D] there
        float *os = &sm.k[0][0];
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
        if (tx == 0 && rows_here)
#pragma unroll
            for (int i = 0; i < kRPS; ++i) sm.m[ty * kRPS + i] = m[i], sm.l[ty * kRPS + i] = l[i];
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
    return rows <= kOneRows ? kOneRows : rows <= kFewRows ? kFewRows : rows <= kSomeRows ? kSomeRows : kManyRows;
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
    return rt == kOneRows   ? f.template operator()<D, kOneRows>()
           : rt == kFewRows ? f.template operator()<D, kFewRows>()
           : rt == kSomeRows ? f.template operator()<D, kSomeRows>()
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

cudaError_t launch_tree_attn(const abg_tree_attn_args &a, void *ws, bool pdl, cudaStream_t stream) {
    AttnArgs p{};
    p.a = a;
    p.G = static_cast<int>(a.Hq / a.Hkv);
    p.scale2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.D)));
    const bool early = pdl && !capturing(stream);
    return a.type == ABG_SB_F32 ? by_shape(a.D, row_tile(p.G, a.max_span), Go{p, ws, early, pdl, stream})
                                : launch_tree_attn16(p, ws, early, pdl, stream);
}

}  // namespace abg
