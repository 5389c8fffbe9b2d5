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
constexpr int kKT = 64;  // tokens a tile

// Rows of one query tile: 16 where a request has no more, else 64.
constexpr int kFewRows = 16, kManyRows = 64;

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
    static constexpr int kLd = D + 4;  // rows of Q and K start in different banks
    static constexpr int kPLd = kRT + 4;
    static constexpr int kParts = kRT == kFewRows ? 4 : 0;
    float q[kRT][kLd];
    float k[kKT][kLd];
    float v[kKT][D];
    float p[kKT][kPLd];                  // weights, token-major
    float s4[kParts][kKT][kFewRows];     // partial scores of a quarter of the columns each
    float corr[kRT];
    int64_t off[2][kKT];                 // a tile's row offsets in elements (-1: none)
    float m[kRT], l[kRT];
    AttnScan scan;
    uint32_t bad[ABG_MAX_SPAN / 32];     // drafts whose V holds an infinity or a NaN
};

// Thread i < kKT: where token i of tile t lies (in elements of its tensor), -1: nowhere.
template <int D>
__device__ __forceinline__ int64_t row_offset(const abg_tree_attn_args &a, const AttnSeg &s, int t, int i) {
    if (t < s.ctiles) {
        const int key = t * kKT + i;
        if (key >= s.req.len) return -1;
        const int j = static_cast<int>(key / static_cast<unsigned>(a.page));
        const int64_t id = a.table[static_cast<int64_t>(s.b) * a.width + j];
        if (id < 0 || id >= a.pages) return -1;
        return ((id * a.Hkv + s.h) * a.page + (key - static_cast<int64_t>(j) * a.page)) * D;
    }
    const int key = (t - s.ctiles) * kKT + i;
    return key < s.req.T ? (s.h * a.drafts + s.req.n0 + key) * static_cast<int64_t>(D) : -1;
}

template <int D>
__device__ __forceinline__ void load_tile(float *dst, int ld, const float *src, const int64_t *off) {
    for (int i = threadIdx.x; i < kKT * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        const int64_t o = off[r];
        cp16(dst + r * ld + c, src + max(o, int64_t(0)) + c, o >= 0);
    }
    cp_commit();
}

// One part of the work line.  Thread (ty, tx) = (tid / 16, tid % 16) holds the
// scores of kRPS rows and tokens tx + 16 j; for the sums, a thread holds four
// columns of kRPO rows over every kKS-th token.
template <int D, int kRT>
__global__ void __launch_bounds__(kThreads) attn_kernel(const __grid_constant__ AttnArgs p) {
    using S = Smem<D, kRT>;
    extern __shared__ __align__(16) unsigned char raw[];
    S &sm = *reinterpret_cast<S *>(raw);
    const abg_tree_attn_args &a = p.a;
    constexpr int kRPS = kRT / 16;
    constexpr int kRPO = kRT == kFewRows ? 4 : 16;
    constexpr int kQuads = D / 4, kRG = kRT / kRPO, kKS = kThreads / (kQuads * kRG);
    constexpr int E = D / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tx = tid % 16, ty = tid / 16;
    const int quad = tid % kQuads, rg = tid / kQuads % kRG, ks = tid / (kQuads * kRG);
    grid_dep_wait();
    grid_dep_launch();
    AttnLine<kRT, kKT> line;
    line.template init<kThreads>(p, blockIdx.x, gridDim.x, sm.scan);
    bool left = false;
    AttnSeg s;
    while (line.next(p, s)) {
        const float *kt, *vt;
        auto source = [&](int t) {
            const bool cache = t < s.ctiles;
            kt = static_cast<const float *>(cache ? a.Kc : a.Kd);
            vt = static_cast<const float *>(cache ? a.Vc : a.Vd);
        };
        __syncthreads();  // the last stretch's shared memory is done with
        for (int i = tid; i < kRT * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4)), row = s.r0 + r;
            float4 v = make_float4(0, 0, 0, 0);
            if (r < s.rows)
                v = *reinterpret_cast<const float4 *>(
                    static_cast<const float *>(a.q) +
                    ((static_cast<int64_t>(s.req.n0) + row / p.G) * a.Hq + s.h * p.G + row % p.G) * D + c);
            *reinterpret_cast<float4 *>(&sm.q[r][c]) = v;
        }
        if (tid < ABG_MAX_SPAN / 32) sm.bad[tid] = 0;
        if (tid < kKT) sm.off[s.t0 & 1][tid] = row_offset<D>(a, s, s.t0, tid);
        __syncthreads();
        source(s.t0);
        load_tile<D>(&sm.k[0][0], S::kLd, kt, sm.off[s.t0 & 1]);
        load_tile<D>(&sm.v[0][0], D, vt, sm.off[s.t0 & 1]);
        float m[kRPS], l[kRPS], o[kRPO][4];
#pragma unroll
        for (int i = 0; i < kRPS; ++i) m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < kRPO; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        for (int t = s.t0; t < s.t1; ++t) {
            const bool drafts = t >= s.ctiles, more = t + 1 < s.t1;
            if (more && tid < kKT) sm.off[(t + 1) & 1][tid] = row_offset<D>(a, s, t + 1, tid);
            cp_wait<1>();
            __syncthreads();
            // scores
            float sc[kRPS][4];
            if constexpr (kRT == kFewRows) {
                // a quarter of the columns of one token a thread, against all rows
                const int key = tid % kKT, part = tid / kKT;
                float acc[kFewRows];
#pragma unroll
                for (int r = 0; r < kFewRows; ++r) acc[r] = 0.0f;
#pragma unroll 2
                for (int c = part * (D / 4); c < (part + 1) * (D / 4); c += 4) {
                    const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[key][c]);
#pragma unroll
                    for (int r = 0; r < kFewRows; ++r) {
                        const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[r][c]);
                        acc[r] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, acc[r]))));
                    }
                }
#pragma unroll
                for (int r = 0; r < kFewRows; r += 4)
                    *reinterpret_cast<float4 *>(&sm.s4[part][key][r]) =
                        make_float4(acc[r], acc[r + 1], acc[r + 2], acc[r + 3]);
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = tx + 16 * j;
                    sc[0][j] = (sm.s4[0][k][ty] + sm.s4[1][k][ty]) + (sm.s4[2][k][ty] + sm.s4[3][k][ty]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kRPS; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.0f;
#pragma unroll 2
                for (int c = 0; c < D; c += 4) {
                    float4 kv[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][c]);
#pragma unroll
                    for (int i = 0; i < kRPS; ++i) {
                        const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[ty * kRPS + i][c]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sc[i][j] = fmaf(qv.x, kv[j].x, fmaf(qv.y, kv[j].y, fmaf(qv.z, kv[j].z,
                                                                                   fmaf(qv.w, kv[j].w, sc[i][j]))));
                    }
                }
                __syncthreads();
            }
            if (more) {
                source(t + 1);
                load_tile<D>(&sm.k[0][0], S::kLd, kt, sm.off[(t + 1) & 1]);
            } else {
                cp_commit();
            }
            // softmax statistics and weights
#pragma unroll
            for (int i = 0; i < kRPS; ++i) {
                const int r = ty * kRPS + i;
                const uint64_t *seen = nullptr;
                if (drafts && r < s.rows)
                    seen = a.mask + (static_cast<int64_t>(s.req.n0) + (s.r0 + r) / p.G) * a.words;
                float top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = (drafts ? t - s.ctiles : t) * kKT + tx + 16 * j;
                    const bool in = drafts ? k < s.req.T && seen && attn_sees(seen, k) : k < s.req.len;
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
                    const float e = exp2f(sc[i][j] - ref);
                    sum += e;
                    sm.p[tx + 16 * j][r] = e;
                }
#pragma unroll
                for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                l[i] = l[i] * corr + sum;
                m[i] = top;
                if (tx == 0) sm.corr[r] = corr;
            }
            cp_wait<1>();
            __syncthreads();
            if (drafts) {
                // an infinity or a NaN in a draft's V must not reach the rows
                // that do not see it (0 * NaN): taken out here, and added at the
                // end to the rows that do
                for (int i = tid; i < kKT * D; i += kThreads) {
                    const int r = i / D;
                    float &v = sm.v[r][i % D];
                    if (!(fabsf(v) < INFINITY)) {
                        v = 0.0f;
                        const int k = (t - s.ctiles) * kKT + r;
                        atomicOr(&sm.bad[k >> 5], 1u << (k & 31));
                    }
                }
                __syncthreads();
            }
            // weighted sums
#pragma unroll
            for (int i = 0; i < kRPO; ++i) {
                const float f = sm.corr[rg * kRPO + i];
                o[i][0] *= f, o[i][1] *= f, o[i][2] *= f, o[i][3] *= f;
            }
#pragma unroll 2
            for (int k = ks; k < kKT; k += kKS) {
                const float4 v = *reinterpret_cast<const float4 *>(&sm.v[k][4 * quad]);
#pragma unroll
                for (int i = 0; i < kRPO; i += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(&sm.p[k][rg * kRPO + i]);
                    const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        o[i + h][0] = fmaf(ww[h], v.x, o[i + h][0]);
                        o[i + h][1] = fmaf(ww[h], v.y, o[i + h][1]);
                        o[i + h][2] = fmaf(ww[h], v.z, o[i + h][2]);
                        o[i + h][3] = fmaf(ww[h], v.w, o[i + h][3]);
                    }
                }
            }
            __syncthreads();
            if (more) {
                load_tile<D>(&sm.v[0][0], D, vt, sm.off[(t + 1) & 1]);
            } else {
                cp_commit();
            }
        }
        cp_wait<0>();
        // the token groups' sums, through the K tile's memory: [kRT][D]
        float *os = &sm.k[0][0];
        for (int g = 0; g < kKS; ++g) {
            if (ks == g)
#pragma unroll
                for (int i = 0; i < kRPO; ++i) {
                    float4 *at = reinterpret_cast<float4 *>(os + (rg * kRPO + i) * D + 4 * quad);
                    float4 v = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                    if (g > 0) {
                        const float4 u = *at;
                        v = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
                    }
                    *at = v;
                }
            __syncthreads();
        }
        if (tx == 0)
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
            for (int k = 0; k < s.req.T; ++k)
                if (sm.bad[k >> 5] >> (k & 31) & 1 && attn_sees(a.mask + n * a.words, k)) {
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

int row_tile(int64_t G, int64_t max_span) { return G * max_span <= kFewRows ? kFewRows : kManyRows; }

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

template <int D>
size_t bytes_of(int rt) {
    return attn_layout(rt == kFewRows ? grid_of<D, kFewRows>() : grid_of<D, kManyRows>(), rt, D).total;
}
template <int D>
cudaError_t go_rows(const AttnArgs &p, int rt, void *ws, bool early, bool pdl, cudaStream_t stream) {
    return rt == kFewRows ? go<D, kFewRows>(p, ws, early, pdl, stream) : go<D, kManyRows>(p, ws, early, pdl, stream);
}

}  // namespace

size_t tree_attn_bytes(int Hq, int Hkv, int D, int max_span, int type) {
    if (type != ABG_SB_F32) return tree_attn16_bytes(D);
    const int rt = row_tile(Hq / Hkv, max_span);
    return D == 64 ? bytes_of<64>(rt) : D == 128 ? bytes_of<128>(rt) : bytes_of<256>(rt);
}

cudaError_t launch_tree_attn(const abg_tree_attn_args &a, void *ws, bool pdl, cudaStream_t stream) {
    AttnArgs p{};
    p.a = a;
    p.G = static_cast<int>(a.Hq / a.Hkv);
    p.scale2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.D)));
    const bool early = pdl && !capturing(stream);
    if (a.type != ABG_SB_F32) return launch_tree_attn16(p, ws, early, pdl, stream);
    const int rt = row_tile(p.G, a.max_span);
    return a.D == 64    ? go_rows<64>(p, rt, ws, early, pdl, stream)
           : a.D == 128 ? go_rows<128>(p, rt, ws, early, pdl, stream)
                        : go_rows<256>(p, rt, ws, early, pdl, stream);
}

}  // namespace abg
