// Shared by the tree_attn kernels: the split of a call's work over the grid,
// what a row's result goes through, and the layout of the workspace.
//
// Work.  The T*G query rows (draft t, head g) of one request that share a
// key/value head are cut into tiles of kRT rows; a unit is such a tile, and its
// work is the kKT-token tiles of the request's cache followed by those of its
// drafts.  The tiles of all units form one line, in request, head, row-tile,
// token order, and block c of C takes its c-th equal part: lengths may be as
// ragged as they like, no block has more than one tile more than another, and
// nothing has to be known on the host.  A part may begin or end inside a unit;
// the unit's pieces then leave their unnormalized sums, maxima and weights in
// the workspace and a second launch joins them, in block order, so that the
// result does not depend on timing.
#pragma once

#include "abg_dev.cuh"
#include "draft.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

namespace abg {

// A unit that ends in another block than it began in, left by the block it
// began in (rows 0: none).
struct AttnSplit {
    int n0;     // first draft row of the request
    int h;      // key/value head
    int r0;     // first row of the unit's tile
    int rows;   // its rows
    int first;  // block it begins in
    int last;   // block it ends in
};

struct AttnArgs {
    abg_tree_attn_args a;
    int G;
    float scale2;  // log2(e) / sqrt(D): scores are kept in base 2
    // workspace: per block two pieces (0: of a unit begun earlier, 1: of a
    // unit that goes on) of kRT rows
    float *part_o;    // [C][2] pieces of kRT * D (attn_piece_at)
    float2 *part_ml;  // [C][2][kRT]  (maximum, weight sum)
    // per unit, or per block where a call may have more units than blocks
    AttnSplit *split;
    int units;      // entries of split
    int per_head;   // entries a (request, head) has; 0: entry c is block c's
};

// A call has at most B * Hkv * per_head units, where a request's rows fill at
// most per_head tiles.  If that is no more than the blocks, a unit's entry is
// its own; otherwise it is that of the block that it begins in.
inline void attn_entries(AttnArgs &p, int C, int rt) {
    const int64_t per_head = (64 * p.a.words * p.G + rt - 1) / rt, units = p.a.B * p.a.Hkv * per_head;
    p.per_head = p.a.B <= C && p.a.Hkv <= C && units <= C ? static_cast<int>(per_head) : 0;
    p.units = p.per_head ? static_cast<int>(units) : C;
}

struct AttnLayout {
    size_t o, ml, split, total;
};
constexpr int kMaxBlocks = 1024;  // of the first launch
inline AttnLayout attn_layout(int C, int rt, int D) {
    AttnLayout l;
    l.o = 0;
    l.ml = static_cast<size_t>(C) * 2 * rt * D * sizeof(float);
    l.split = l.ml + static_cast<size_t>(C) * 2 * rt * sizeof(float2);
    l.total = l.split + static_cast<size_t>(C) * sizeof(AttnSplit);
    return l;
}

// --------------------------------------------------------- the work line ---
struct AttnReq {
    int n0, T, len;  // first draft row, drafts, cached tokens
};
__device__ __forceinline__ AttnReq attn_req(const abg_tree_attn_args &a, int b) {
    AttnReq r;
    r.n0 = max(0, a.cu[b]);
    const int64_t hi = min(a.N, static_cast<int64_t>(a.cu[b + 1]));
    r.T = static_cast<int>(max(int64_t(0), min(hi - r.n0, 64 * a.words)));
    r.len = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(a.lens[b]), a.width * a.page)));
    return r;
}

template <int kRT, int kKT>
__device__ __forceinline__ int64_t attn_weight(const AttnArgs &p, const AttnReq &r) {
    const int64_t units = p.a.Hkv * ((static_cast<int64_t>(r.T) * p.G + kRT - 1) / kRT);
    return units * ((static_cast<uint32_t>(r.len) + kKT - 1) / kKT + (r.T + kKT - 1) / kKT);
}

// a / b of nonnegative numbers; 64-bit division is a long subroutine, and the
// line of all but enormous calls fits in 32 bits.
__device__ __forceinline__ int64_t attn_div(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// One stretch of a unit's token tiles.
struct AttnSeg {
    AttnReq req;
    int b, h, r0, rows;      // request, head, first row and rows of the unit
    int ctiles, tiles;       // cache tiles, all tiles of the unit
    int t0, t1;              // the stretch
    int64_t unit;            // the unit's place on the line
};

// Shared memory of AttnLine::init.
struct AttnScan {
    int64_t w[32], ex;
    int b;
};

// A block's part of the line; every thread holds the same values.
template <int kRT, int kKT>
struct AttnLine {
    int64_t W, cur, end, ex;  // all tiles; this block's rest; place of request b
    int b, C;                 // request; blocks that have a part

    // By a whole block of kThreads threads: part c of the line.  Blocks get at
    // least two tiles each, so that a short call is not all joining.
    template <int kThreads>
    __device__ __forceinline__ void init(const AttnArgs &p, int c, int grid, AttnScan &sm) {
        const int tid = threadIdx.x, lane = tid & 31;
        const int B = static_cast<int>(p.a.B);
        if (B <= 32) {  // every warp for itself
            int64_t x = lane < B ? attn_weight<kRT, kKT>(p, attn_req(p.a, lane)) : 0;
            const int64_t w = x;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += u;
            }
            part(__shfl_sync(0xffffffffu, x, 31), c, grid);
            const unsigned here = __ballot_sync(0xffffffffu, x - w <= cur && cur < x);
            b = here ? __ffs(static_cast<int>(here)) - 1 : B;
            ex = __shfl_sync(0xffffffffu, x - w, b & 31);
        } else {
            scan<kThreads>(p, c, grid, sm);
        }
    }

    __device__ __forceinline__ void part(int64_t all, int c, int grid) {
        W = all;
        C = static_cast<int>(min(static_cast<int64_t>(grid), max(int64_t(1), W / 2)));
        cur = c < C ? attn_div(W * c, C) : W;
        end = c < C ? attn_div(W * (c + 1), C) : W;
    }

    template <int kThreads>
    __device__ __forceinline__ void scan(const AttnArgs &p, int c, int grid, AttnScan &sm) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int B = static_cast<int>(p.a.B);
        const int64_t w0 = tid < B ? attn_weight<kRT, kKT>(p, attn_req(p.a, tid)) : 0;
        int64_t sum = w0;
        for (int i = kThreads + tid; i < B; i += kThreads) sum += attn_weight<kRT, kKT>(p, attn_req(p.a, i));
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) sm.w[warp] = sum;
        if (tid == 0) sm.b = B;
        __syncthreads();
        sum = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) sum += sm.w[w];
        part(sum, c, grid);
        ex = 0;
        b = B;
        if (cur >= end) return;  // uniform
        int64_t before = 0;
        for (int b0 = 0; b0 < B; b0 += kThreads) {
            const int i = b0 + tid;
            const int64_t w = b0 == 0 ? w0 : i < B ? attn_weight<kRT, kKT>(p, attn_req(p.a, i)) : 0;
            int64_t x = w;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += u;
            }
            __syncthreads();  // sm.w's last readers are done
            if (lane == 31) sm.w[warp] = x;
            __syncthreads();
            int64_t all = 0;
#pragma unroll
            for (int v = 0; v < kThreads / 32; ++v) {
                if (v == warp) x += before + all;
                all += sm.w[v];
            }
            before += all;
            if (i < B && x - w <= cur && cur < x) sm.b = i, sm.ex = x - w;
            __syncthreads();
            if (sm.b < B) break;
        }
        b = sm.b;
        ex = sm.ex;
    }

    // The next stretch (false: the part is done).
    __device__ __forceinline__ bool next(const AttnArgs &p, AttnSeg &s) {
        if (cur >= end) return false;
        int64_t w;
        for (;; ++b, ex += w) {
            s.req = attn_req(p.a, b);
            w = attn_weight<kRT, kKT>(p, s.req);
            if (cur - ex < w) break;
        }
        const int R = s.req.T * p.G, nrt = (R + kRT - 1) / kRT;
        s.ctiles = static_cast<int>((static_cast<uint32_t>(s.req.len) + kKT - 1) / kKT);
        s.tiles = s.ctiles + (s.req.T + kKT - 1) / kKT;
        const int64_t u = attn_div(cur - ex, s.tiles);
        s.unit = ex + u * s.tiles;
        s.t0 = static_cast<int>(cur - s.unit);
        s.t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), s.t0 + (end - cur)));
        s.b = b;
        s.h = static_cast<int>(u / nrt);
        s.r0 = static_cast<int>(u - static_cast<int64_t>(s.h) * nrt) * kRT;
        s.rows = min(kRT, R - s.r0);
        cur += s.t1 - s.t0;
        return true;
    }

    // where a unit that begins in this block leaves what it is
    __device__ __forceinline__ AttnSplit *entry(const AttnArgs &p, const AttnSeg &s, int c) const {
        return p.split +
               (p.per_head ? (static_cast<int64_t>(s.b) * p.a.Hkv + s.h) * p.per_head + s.r0 / kRT : int64_t(c));
    }
    // By one thread, once a stretch: says whether and where the unit that
    // begins here goes on.  Units in one block have an entry too where entries
    // are per unit (nothing else writes it).
    __device__ __forceinline__ void leave_entry(const AttnArgs &p, const AttnSeg &s, int c, bool &left) const {
        if (s.t0 != 0) return;
        AttnSplit sp{};
        if (s.t1 < s.tiles) {
            // the block that holds the unit's last tile
            const int last = static_cast<int>(attn_div((s.unit + s.tiles) * C + W - 1, W) - 1);
            sp = AttnSplit{s.req.n0, s.h, s.r0, s.rows, c, last};
            left = true;
        }
        if (p.per_head || s.t1 < s.tiles) *entry(p, s, c) = sp;
    }
    // By the same thread at the end: a block's entry says so if there is none.
    __device__ __forceinline__ void end_entries(const AttnArgs &p, int c, bool left) const {
        if (!p.per_head && !left) p.split[c] = AttnSplit{};
    }
};

// Whether draft t of the request (mask row m) sees draft j.
__device__ __forceinline__ bool attn_sees(const uint64_t *m, int j) { return m[j >> 6] >> (j & 63) & 1; }

// ------------------------------------------------------------- the result --
// By a warp, lane l holding columns l*D/32 ..: one row's sums o and weight l
// become y (gate, group sums).
template <typename T>
__device__ __forceinline__ T attn_round(float v) {
    if constexpr (std::is_same_v<T, float>) {
        return v;
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        return __float2bfloat16_rn(v);
    } else {
        return __float2half_rn(v);
    }
}

template <typename T, int D>
__device__ __forceinline__ void attn_finish(const abg_tree_attn_args &a, int64_t n, int hq, const float (&o)[D / 32],
                                            float l) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t at = (n * a.Hq + hq) * D + lane * E;
    float v[E], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        v[i] = l == 0.0f ? 0.0f : o[i] / l;
        if (a.gate) v[i] *= 1.0f / (1.0f + expf(-a.gate[at + i]));
    }
    if (a.y_type == ABG_SB_F32) {
        float *y = static_cast<float *>(a.y) + at;
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = v[i];
    } else {
        T *y = static_cast<T *>(a.y) + at;
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = attn_round<T>(v[i]);
    }
    if (a.ysum) {
#pragma unroll
        for (int i = 0; i < E; ++i) sum += v[i];
#pragma unroll
        for (int d = 1; d < 64 / E; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane % (64 / E) == 0) a.ysum[at / 64] = sum;
    }
}

// Where four columns 4q .. 4q+3 of row r of a piece lie (in floats).  The
// kernel with a thread a row writes them quad by quad with the rows side by
// side (kByQuad), the one with a warp a row writes whole rows.
template <int D, int kRT, bool kByQuad>
__device__ __forceinline__ int64_t attn_piece_at(int64_t piece, int r, int q) {
    return kByQuad ? ((piece * (D / 4) + q) * kRT + r) * 4 : (piece * kRT + r) * D + 4 * q;
}

// Joins the pieces of split units: block (u, y) the rows y * 8/kWarps .. of
// entry u, kWarps warps a row.  A warp takes every kWarps-th piece, with a
// running maximum (so that no load waits for another), and the warps of a row
// meet in shared memory.  Latency bounds it: the pieces of 152 blocks, of 96 rows
// of 128 columns, take 11.7 us on their own out of memory, of 256 rows 13.9; after
// the first launch, out of the second-level cache, 3-5.
template <typename T, int D, int kRT, bool kByQuad, int kWarps, int kBatch>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnArgs p) {
    constexpr int E = D / 32, kRows = 8 / kWarps;
    __shared__ __align__(16) float s_o[8][D];
    __shared__ float2 s_ml[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kWarps;
    grid_dep_wait();
    grid_dep_launch();
    AttnSplit s = p.split[blockIdx.x];
    if (p.per_head) {  // a request without drafts, or a tile past its rows, has no entry
        const int64_t per = p.a.Hkv * p.per_head;
        const int b = static_cast<int>(blockIdx.x / per);
        if (static_cast<int64_t>(attn_req(p.a, b).T) * p.G <= static_cast<int64_t>(blockIdx.x % p.per_head) * kRT) return;
    }
    // piece k of the unit: the first block's second piece, then the first pieces of the others
    const int pieces = s.last - s.first + 1;
    for (int r0 = blockIdx.y * kRows; r0 < s.rows; r0 += gridDim.y * kRows) {
        const int r = r0 + warp / kWarps;
        float m = -INFINITY, L = 0.0f, o[E] = {};
        if (r < s.rows) {
            for (int k0 = sub; k0 < pieces; k0 += kBatch * kWarps) {
                float2 ml[kBatch];
                float v[kBatch][E];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int k = k0 + u * kWarps;
                    ml[u] = make_float2(-INFINITY, 0.0f);
                    if (k >= pieces) continue;
                    const int64_t piece = static_cast<int64_t>(2) * (s.first + k) + (k == 0);
                    ml[u] = p.part_ml[piece * kRT + r];
                    if constexpr (E == 2) {
                        const float2 x = *reinterpret_cast<const float2 *>(
                            p.part_o + attn_piece_at<D, kRT, kByQuad>(piece, r, lane / 2) + 2 * (lane & 1));
                        v[u][0] = x.x, v[u][1] = x.y;
                    } else {
#pragma unroll
                        for (int q = 0; q < E / 4; ++q) {
                            const float4 x = *reinterpret_cast<const float4 *>(
                                p.part_o + attn_piece_at<D, kRT, kByQuad>(piece, r, lane * (E / 4) + q));
                            v[u][4 * q] = x.x, v[u][4 * q + 1] = x.y, v[u][4 * q + 2] = x.z, v[u][4 * q + 3] = x.w;
                        }
                    }
                }
                float top = m;
#pragma unroll
                for (int u = 0; u < kBatch; ++u) top = fmaxf(top, ml[u].x);
                const float ref = top == -INFINITY ? 0.0f : top, f = exp2f(m - ref);
                m = top;
                L *= f;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    if (ml[u].y == 0.0f) continue;  // no weight: nothing to add, not a NaN either
                    const float w = exp2f(ml[u].x - ref);
                    L += ml[u].y * w;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] += v[u][e] * w;
                }
            }
        }
        if constexpr (kWarps > 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
            if (lane == 0) s_ml[warp] = make_float2(m, L);
            __syncthreads();
            if (sub == 0) {
                float top = m;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_ml[warp + w].x);
                const float ref = top == -INFINITY ? 0.0f : top;
                const float f = L == 0.0f ? 0.0f : exp2f(m - ref);
                L *= f;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] *= f;  // (without weight o is 0; a NaN stays, as infinity * 0)
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float2 ml = s_ml[warp + w];
                    if (ml.y == 0.0f) continue;
                    const float g = exp2f(ml.x - ref);
                    L += ml.y * g;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] += s_o[warp + w][lane * E + e] * g;
                }
            }
        }
        if (r < s.rows && sub == 0) {
            const int row = s.r0 + r;
            attn_finish<T, D>(p.a, static_cast<int64_t>(s.n0) + row / p.G, s.h * p.G + row % p.G, o, L);
        }
        if constexpr (kWarps > 1) __syncthreads();
    }
}

// The joining launch, early (it waits for the first).  Few units are many
// pieces each: more warps a row.  kBatch: pieces that a warp loads at a time.
template <typename T, int D, int kRT, bool kByQuad, int kBatch = 4>
cudaError_t launch_join(const AttnArgs &p, int C, bool pdl, cudaStream_t stream) {
    const int64_t units = p.per_head ? p.units : C, span_rows = p.a.max_span * p.G;
    const int64_t rows = std::min<int64_t>(kRT, span_rows);
    const int64_t filled = p.a.B * p.a.Hkv * ((span_rows + kRT - 1) / kRT);  // units with rows, of spans as told
    const int64_t pieces = C / std::max<int64_t>(1, filled) + 1;
    auto go = [&](auto w) {
        constexpr int kWarps = decltype(w)::value;
        const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>((rows * kWarps + 7) / 8));
        return launch_kernel(attn_join_kernel<T, D, kRT, kByQuad, kWarps, kBatch>, grid, dim3(256), 0, stream, pdl, p);
    };
    return pieces > 32  ? go(std::integral_constant<int, 8>{})
           : pieces > 6 ? go(std::integral_constant<int, 4>{})
                        : go(std::integral_constant<int, 1>{});
}

}  // namespace abg
