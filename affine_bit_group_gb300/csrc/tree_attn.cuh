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

namespace abg {

// A unit that ends in another block than it began in, left by the block it
// began in (rows 0: none).
struct AttnSplit {
    int n0;    // first draft row of the request
    int h;     // key/value head
    int r0;    // first row of the unit's tile
    int rows;  // its rows
    int last;  // block it ends in
};

struct AttnArgs {
    abg_tree_attn_args a;
    int G;
    float scale2;  // log2(e) / sqrt(D): scores are kept in base 2
    // workspace: per block two pieces (0: of a unit begun earlier, 1: of a
    // unit that goes on) of kRT rows
    float *part_o;    // [C][2] pieces of kRT * D (attn_piece_at)
    float2 *part_ml;  // [C][2][kRT]  (maximum, weight sum)
    AttnSplit *split;  // [C]
};

struct AttnLayout {
    size_t o, ml, split, total;
};
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
    return units * ((static_cast<int64_t>(r.len) + kKT - 1) / kKT + (r.T + kKT - 1) / kKT);
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
    __device__ void init(const AttnArgs &p, int c, int grid, AttnScan &sm) {
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
        W = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) W += sm.w[w];
        C = static_cast<int>(min(static_cast<int64_t>(grid), max(int64_t(1), W / 2)));
        cur = c < C ? W * c / C : W;
        end = c < C ? W * (c + 1) / C : W;
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
        s.ctiles = (s.req.len + kKT - 1) / kKT;
        s.tiles = s.ctiles + (s.req.T + kKT - 1) / kKT;
        const int64_t u = (cur - ex) / s.tiles;
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

    __device__ __forceinline__ int block_of_end(int64_t e) const {  // block that holds tile e-1
        return static_cast<int>((e * C + W - 1) / W - 1);
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

// Joins the pieces of split units.  The rows of all split units are dealt out
// to all blocks (few units may hold all of them): eight rows a block, a warp
// each, where a unit has up to eight pieces; else one row a block, whose warps
// take every eighth piece each and meet in shared memory.
constexpr int kJoinWarps = 8;

__device__ __forceinline__ int join_tasks(const AttnSplit &s, int c) {
    return s.last - c < kJoinWarps ? (s.rows + kJoinWarps - 1) / kJoinWarps : s.rows;
}
constexpr int kJoinMax = 1024;  // split units at most (one a block of the first launch)

template <typename T, int D, int kRT, bool kByQuad>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const __grid_constant__ AttnArgs p, int C) {
    constexpr int E = D / 32, kThreads = 32 * kJoinWarps;
    __shared__ int s_upto[kJoinMax];  // tasks of units 0 .. c
    __shared__ int s_warp[kJoinWarps];
    __shared__ __align__(16) float s_o[kJoinWarps][D];
    __shared__ float s_l[kJoinWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_wait();
    int total = 0;
    for (int c0 = 0; c0 < C; c0 += kThreads) {
        const int c = c0 + tid;
        int x = c < C ? join_tasks(p.split[c], c) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += u;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            if (w == warp) x += total + all;
            all += s_warp[w];
        }
        total += all;
        if (c < C) s_upto[c] = x;
        __syncthreads();
    }
    for (int i = blockIdx.x; i < total; i += gridDim.x) {
        int lo = 0, hi = C - 1;  // the first unit with upto > i
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_upto[mid] > i) {
                hi = mid;
            } else {
                lo = mid + 1;
            }
        }
        const AttnSplit s = p.split[lo];
        const int task = i - (lo ? s_upto[lo - 1] : 0);
        // piece k of the unit: block lo's second piece, then the first pieces of lo+1 .. last
        const int pieces = s.last - lo + 1;
        const bool few = pieces <= kJoinWarps;
        const int r = few ? task * kJoinWarps + warp : task;
        if (few && r >= s.rows) continue;  // no barrier follows
        auto piece = [&](int k) { return static_cast<int64_t>(2) * (lo + k) + (k == 0); };
        float M = -INFINITY;
        for (int k = lane; k < pieces; k += 32) M = fmaxf(M, p.part_ml[piece(k) * kRT + r].x);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        if (M == -INFINITY) M = 0.0f;
        float o[E] = {}, L = 0.0f;
#pragma unroll 4
        for (int k = few ? 0 : warp; k < pieces; k += few ? 1 : kJoinWarps) {
            const float2 ml = p.part_ml[piece(k) * kRT + r];
            const float w = exp2f(ml.x - M);
            L += ml.y * w;
            if constexpr (E == 2) {
                const float2 v = *reinterpret_cast<const float2 *>(
                    p.part_o + attn_piece_at<D, kRT, kByQuad>(piece(k), r, lane / 2) + 2 * (lane & 1));
                o[0] += ml.y == 0.0f ? 0.0f : v.x * w, o[1] += ml.y == 0.0f ? 0.0f : v.y * w;
            } else {
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    const float4 v = *reinterpret_cast<const float4 *>(
                        p.part_o + attn_piece_at<D, kRT, kByQuad>(piece(k), r, lane * (E / 4) + q));
                    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[4 * q + e] += ml.y == 0.0f ? 0.0f : x[e] * w;
                }
            }
        }
        if (!few) {
#pragma unroll
            for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
            if (lane == 0) s_l[warp] = L;
            __syncthreads();
            if (warp == 0)
                for (int w = 1; w < kJoinWarps; ++w) {
                    L += s_l[w];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] += s_o[w][lane * E + e];
                }
        }
        if (few || warp == 0) {
            const int row = s.r0 + r;
            attn_finish<T, D>(p.a, static_cast<int64_t>(s.n0) + row / p.G, s.h * p.G + row % p.G, o, L);
        }
        if (!few) __syncthreads();
    }
}

// Blocks of the joining launch: about as many as fit at once.
constexpr int kJoinBlocksPerSm = 4;

}  // namespace abg
