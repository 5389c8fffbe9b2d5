// Planning, cache layout and acceptance of drafted tokens: page_plan,
// tree_plan, kv_put and tree_accept (their formulas are in include/abg.h).
//
// The norm and rotation of kv_put are the steps of the single-token attention
// ("Metal: queued rmsq, swq, gdn and atq kernels ...", bendlang/bend #1440,
// Change, the Array.atq bullet); the rest has no counterpart on the pages.
#include "abg_dev.cuh"
#include "abg_kernels.cuh"
#include "draft.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

namespace abg {

namespace {

// ---------------------------------------------------------- page_plan ------
// One launch: every block scans all requests (a few loads a thread: at most
// 8192 requests) and keeps each one's place in the ring in shared memory, so
// that no block waits for another; the first blocks then share the tokens, the
// others the tables (a warp a request).  A token of a fresh page takes the page
// from the ring itself, not from the table entry that another block writes.
// Latency bounds it: 384 tokens of 48 requests take 5 us (3 of them from launch
// to launch), 768000 tokens of 512 requests 10.3 us, 0.9 TB/s.
constexpr int kPlanThreads = 512;

// Entry i of the ring, 0 <= i < 2^62, from an entry `base` in 0 .. len-1 on.
__device__ __forceinline__ int ring_at(int base, int64_t i, int len) {
    const int64_t at = base + i;
    return static_cast<int>(at < len ? at : at < 2ll * len ? at - len : at % len);
}

struct Ask {
    int64_t total, extra, freed;
    bool gone, bad;
};

__device__ __forceinline__ Ask ask_of(const PagePlanArgs &a, int b) {
    Ask k;
    const int64_t len = a.lens[b], add = a.add[b];
    const int held = a.held[b];
    const int64_t span = static_cast<int64_t>(a.cu[b + 1]) - a.cu[b];
    k.gone = add < 0;
    k.total = len + add;
    k.bad = len < 0 || held < 0 || held > a.width;
    int need = 0;
    if (!k.gone && !k.bad) {
        k.bad = add > span || k.total > 0x7fffffff;
        if (!k.bad) {
            need = static_cast<int>((static_cast<uint32_t>(k.total) + static_cast<uint32_t>(a.page - 1)) /
                                    static_cast<uint32_t>(a.page));
            k.bad = need > a.width;
        }
    }
    k.extra = k.gone || k.bad ? 0 : max(0, need - held);
    k.freed = k.gone && !k.bad ? held : 0;
    return k;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PagePlanArgs a,
                                                                 int token_blocks) {
    extern __shared__ int32_t sm[];
    int32_t *s_cu = sm;              // [B+1]
    int32_t *s_at = sm + a.B + 1;    // [B] ring entry of the first fresh or freed page; -1: refused
    __shared__ int64_t s_sum[2][kPlanThreads / 32];
    __shared__ int s_bad[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.pos)) & 15) == 0;
    const int64_t head = a.ends[0], tail = a.ends[1];
    const int64_t avail = max(int64_t(0), min(tail - head, static_cast<int64_t>(a.ring_len)));
    const int R = a.ring_len;
    const int64_t room = R - avail;  // pages given back never lie over free ones, which others read meanwhile
    const int head0 = static_cast<int>((head % R + R) % R), tail0 = static_cast<int>((tail % R + R) % R);
    int64_t done_x = 0, done_f = 0;
    int64_t taken = 0, given = 0;  // extras up to the last request that was granted any, pages up to the last given back
    int bad = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        Ask k{};
        if (b < a.B) {
            k = ask_of(a, b);
            s_cu[b] = a.cu[b];
        }
        int64_t x = k.extra, f = k.freed;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t ux = __shfl_up_sync(0xffffffffu, x, d), uf = __shfl_up_sync(0xffffffffu, f, d);
            if (lane >= d) x += ux, f += uf;
        }
        if (lane == 31) s_sum[0][warp] = x, s_sum[1][warp] = f;
        __syncthreads();
        int64_t all_x = 0, all_f = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w == warp) x += done_x + all_x, f += done_f + all_f;
            all_x += s_sum[0][w], all_f += s_sum[1][w];
        }
        done_x += all_x, done_f += all_f;
        if (b < a.B) {
            const bool ok = !k.gone && !k.bad && (k.extra == 0 || x <= avail);
            const bool done = k.gone && !k.bad && (k.freed == 0 || f <= room);
            if (ok && k.extra > 0) taken = x;
            if (done && k.freed > 0) given = f;
            bad += !ok && !done;
            s_at[b] = ok ? ring_at(head0, x - k.extra, R) : done ? ring_at(tail0, f - k.freed, R) : -1;
            if (blockIdx.x == 0) {
                const int32_t held = a.held[b];
                a.lens_out[b] = ok ? static_cast<int32_t>(k.total) : done ? 0 : a.lens[b];
                a.held_out[b] = ok ? static_cast<int32_t>(held + k.extra) : done ? 0 : held;
            }
        }
        __syncthreads();
    }
    if (tid == 0) s_cu[a.B] = a.cu[a.B];
    if (blockIdx.x == 0) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, d));
            given = max(given, __shfl_xor_sync(0xffffffffu, given, d));
            bad += __shfl_xor_sync(0xffffffffu, bad, d);
        }
        if (lane == 0) s_sum[0][warp] = taken, s_sum[1][warp] = given, s_bad[warp] = bad;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        for (int w = 1; w < kPlanThreads / 32; ++w)
            taken = max(taken, s_sum[0][w]), given = max(given, s_sum[1][w]), bad += s_bad[w];
        a.ends_out[0] = head + taken;
        a.ends_out[1] = tail + given;
        a.info[0] = static_cast<int32_t>(taken);
        a.info[1] = bad;
    }
    if (static_cast<int>(blockIdx.x) >= token_blocks) {  // table and ring entries
        const int gw = (blockIdx.x - token_blocks) * (kPlanThreads / 32) + warp;
        const int nw = (gridDim.x - token_blocks) * (kPlanThreads / 32);
        for (int b = gw; b < a.B; b += nw) {
            const int at = s_at[b];
            if (at < 0) continue;
            int32_t *row = a.table + static_cast<int64_t>(b) * a.width;
            const Ask k = ask_of(a, b);
            const int held = a.held[b];
            for (int64_t j = lane; j < k.extra; j += 32) row[held + j] = a.ring[ring_at(at, j, R)];
            for (int64_t j = lane; j < k.freed; j += 32) a.ring[ring_at(at, j, R)] = row[j];
        }
        return;
    }
    // slots: a thread four tokens in a row, which mostly share a request and a
    // page, so that the search and the table's latency are paid once for them
    const int64_t quads = (static_cast<int64_t>(a.N) + 3) / 4;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid; i < quads;
         i += static_cast<int64_t>(token_blocks) * kPlanThreads) {
        const int n0 = static_cast<int>(4 * i), end = s_cu[a.B];
        int64_t slot[4];
        int32_t pos[4];
        int b = request_of(s_cu, a.B, n0), page = -1, seen = -1;
        int32_t lo = 0, at = -1, add = 0, len = 0, held = 0, id = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int n = n0 + k;
            slot[k] = -1;
            pos[k] = 0;
            if (n >= end || n >= a.N) continue;
            while (b + 1 < a.B && s_cu[b + 1] <= n) ++b;
            if (b != seen) {
                seen = b;
                page = -1;
                lo = s_cu[b], at = s_at[b], add = a.add[b], len = a.lens[b], held = a.held[b];
            }
            const int t = n - lo;
            if (t < 0 || at < 0 || t >= add) continue;
            pos[k] = len + t;
            const int j = pos[k] / a.page;
            if (j != page) {
                page = j;
                id = j < held ? a.table[static_cast<int64_t>(b) * a.width + j]
                              : a.ring[ring_at(at, j - held, R)];
            }
            slot[k] = static_cast<int64_t>(id) * a.page + (pos[k] - j * a.page);
        }
        if (wide && n0 + 3 < a.N) {
            longlong2 *to = reinterpret_cast<longlong2 *>(a.slots + n0);
            to[0] = make_longlong2(slot[0], slot[1]);
            to[1] = make_longlong2(slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.pos + n0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n0 + k < a.N) a.slots[n0 + k] = slot[k], a.pos[n0 + k] = pos[k];
        }
    }
}

// ---------------------------------------------------------- tree_plan ------
// A block a request, a thread a draft.  Each round a draft joins its pointer's
// mask to its own and moves the pointer to the pointer's pointer, so the
// pointer is 2^r ancestors away after r rounds: log2(span) rounds instead of
// the span's longest chain.  A cycle only repeats bits.  A block a request;
// launching bounds it: 256 spans of up to 120 drafts take 2.5 us from launch to launch.
template <int W>
__global__ void __launch_bounds__(64 * W) tree_plan_kernel(const int32_t *parent, const int32_t *lens,
                                                           const int32_t *cu, uint64_t *mask, int32_t *pos, int B,
                                                           int N) {
    __shared__ uint64_t s_mask[2][W][64 * W];
    __shared__ int16_t s_up[2][64 * W];
    const int b = blockIdx.x, i = threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    const int lo = max(0, b < B ? cu[b] : cu[B]), hi = min(N, b < B ? cu[b + 1] : N);
    const int T = b < B ? max(0, min(hi - lo, 64 * W)) : 0;
    uint64_t m[W];
#pragma unroll
    for (int w = 0; w < W; ++w) m[w] = 0;
    int up = -1;
    bool real = false;
    if (i < T) {
        up = parent[lo + i];
        real = up >= -1;
#pragma unroll
        for (int w = 0; w < W; ++w) m[w] = real && (i >> 6) == w ? 1ull << (i & 63) : 0;
        if (up == i || up >= T) up = -1;
    }
    s_up[1][i] = real ? 0 : -1;  // whether draft i can be an ancestor
    __syncthreads();
    if (up < 0 || s_up[1][up] < 0) up = -1;
    int now = 0;
    for (int reach = 1; reach < T; reach *= 2) {
#pragma unroll
        for (int w = 0; w < W; ++w) s_mask[now][w][i] = m[w];
        s_up[now][i] = static_cast<int16_t>(up);
        if (!__syncthreads_or(up >= 0)) break;
        if (up >= 0) {
#pragma unroll
            for (int w = 0; w < W; ++w) m[w] |= s_mask[now][w][up];
            up = s_up[now][up];
        }
        now ^= 1;
    }
    if (i < T) {
        int depth = -1;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            mask[static_cast<int64_t>(lo + i) * W + w] = m[w];
            depth += __popcll(m[w]);
        }
        pos[lo + i] = real ? lens[b] + depth : 0;
    }
    for (int64_t n = static_cast<int64_t>(lo) + T + i; n < hi; n += 64 * W) {  // padding rows
#pragma unroll
        for (int w = 0; w < W; ++w) mask[n * W + w] = 0;
        pos[n] = 0;
    }
}

// -------------------------------------------------------------- kv_put -----
// A warp a token and 8 of its heads (4 of 256 columns), q heads, then k, then v,
// two at a time: lane l of a half warp holds columns V*l .. V*l+V-1 of a head
// (V = D/32) and the ones D/2 further on, so that the rotation stays in the
// lane.  The squares are summed as the pairwise tree: each half of the columns
// in the lane and over the lanes, then the two halves.  The warps of a full
// grid go through all units, a unit's heads are loaded at once, beside the
// token's rotation and before its slot is looked at, and the next unit's row,
// slot and position are already on their way.  Instructions bound it as much as
// bytes: a lane a column pair, not a lane a column, and the heads' norm factors
// (a division, a root and a reciprocal, each rounded) side by side in the lanes.
// 8191 rows of 16 + 4 + 4 heads of 128, f32 to bf16: 32.7 us for 156 MB, 4.8 TB/s,
// 70% of a plain copy's rate (35.0 without the early start).  A lane a column took
// 53 us.
constexpr int kPutWarps = 8;

template <typename T>
__device__ __forceinline__ float widen(T v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else {
        return static_cast<float>(v);
    }
}
template <typename T>
__device__ __forceinline__ T narrow(float v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        return __float2bfloat16_rn(v);
    } else {
        return __float2half_rn(v);
    }
}

// a / b of nonnegative numbers, in 32 bits where they fit (64-bit division is
// a long subroutine)
__device__ __forceinline__ int64_t div_up_to_64(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// E consecutive values, E * sizeof(T) = 4, 8, 16 or 32 bytes
template <typename T, int E>
__device__ __forceinline__ void load_e(const T *p, float (&v)[E]) {
    constexpr int kBytes = E * sizeof(T);
    alignas(16) T t[E];
    if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t *>(t) = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2 *>(t) = *reinterpret_cast<const uint2 *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            reinterpret_cast<uint4 *>(t)[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = widen(t[i]);
}
template <typename T, int E>
__device__ __forceinline__ void store_e(T *p, const float (&v)[E]) {
    constexpr int kBytes = E * sizeof(T);
    alignas(16) T t[E];
#pragma unroll
    for (int i = 0; i < E; ++i) t[i] = narrow<T>(v[i]);
    if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<uint32_t *>(t);
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(t);
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<uint4 *>(t)[i];
    }
}

template <int D>
struct Put {
    static constexpr int V = D / 32;                    // columns of a chunk
    static constexpr int kSteps = D == 256 ? 2 : 4;
    static constexpr int kHeads = 2 * kSteps;           // of a unit
};

// Pairwise tree of V values.
template <int V>
__device__ __forceinline__ float chunk_tree(const float (&u)[V]) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __fmul_rn(u[i], u[i]);
#pragma unroll
    for (int k = V / 2; k >= 1; k >>= 1)
#pragma unroll
        for (int i = 0; i < k; ++i) x[i] = __fadd_rn(x[2 * i], x[2 * i + 1]);
    return x[0];
}

template <typename S, typename T, int D>
__global__ void __launch_bounds__(32 * kPutWarps, D == 256 ? 2 : D == 128 ? 3 : 4) kv_put_kernel(
    const __grid_constant__ abg_kv_put_args a, int groups) {
    using P = Put<D>;
    constexpr int V = P::V, kSteps = P::kSteps;
    const int lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
    const int64_t units = a.N * groups, stride = static_cast<int64_t>(gridDim.x) * kPutWarps;
    const int nq = a.q ? static_cast<int>(a.Hq) : 0, nk = static_cast<int>(a.Hkv), heads = nq + 2 * nk;
    // (no launch after this one starts early: abg_atq's reads its key cache before it waits)
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
            const bool kept = t.slot >= 0 && t.slot < a.pages * a.page;
            const int64_t page = kept ? div_up_to_64(t.slot, a.page) : 0;
            const int64_t base = page * a.Hkv * a.page + (t.slot - page * a.page);
#pragma unroll
            for (int r = 0; r < kSteps; ++r) {
                const int h = t.h0 + 2 * r + half;
                const float f = __shfl_sync(0xffffffffu, factor, r, 16);
                if (h >= heads || (h >= nq && !kept)) continue;
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
                T *to = h < nq        ? static_cast<T *>(a.qo) + (t.n * a.Hq + h) * D
                        : h < nq + nk ? static_cast<T *>(a.Kc) + (base + (h - nq) * a.page) * D
                                      : static_cast<T *>(a.Vc) + (base + (h - nq - nk) * a.page) * D;
                store_e<T, V>(to + V * l, u[r][0]);
                store_e<T, V>(to + D / 2 + V * l, u[r][1]);
            }
        }
        t = next;
    }
}

// --------------------------------------------------------- tree_accept -----
// The logits are read once, a block a slice of a row; a slice's answer is one
// 64-bit key, the value's order in the upper half and ~index in the lower, so
// that the largest key is the largest value at its lowest index.  Memory bounds
// it: 304 rows of 248320, 302 MB, with accept_kernel in 54.0 us (5.6 TB/s, 83% of a
// plain copy's rate); 8 rows, 7.9 MB, in 6.4 us.
constexpr int kBestThreads = 256;

__device__ __forceinline__ uint64_t best_key(float v, uint32_t i) {
    uint32_t u = __float_as_uint(v != v ? __int_as_float(0xff800000) : v + 0.0f);  // + 0: -0 orders as 0
    u = u & 0x80000000u ? ~u : u | 0x80000000u;
    return static_cast<uint64_t>(u) << 32 | ~i;
}

__global__ void __launch_bounds__(kBestThreads) best_kernel(const float *logits, int64_t ld, int64_t V, int slices,
                                                            int64_t slice, uint64_t *parts) {
    __shared__ uint64_t s_key[kBestThreads / 32];
    const int tid = threadIdx.x;
    const int64_t n = blockIdx.x / slices;
    const float *row = logits + n * ld;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t lo = (blockIdx.x - n * slices) * slice, hi = min(V, lo + slice);
    // whole 16-byte quads from the first aligned element on, single ones around them
    const int64_t off = ((16 - (reinterpret_cast<uintptr_t>(row + lo) & 15)) & 15) / 4;
    const int64_t q0 = min(hi, lo + off), nq = (hi - q0) / 4;
    uint64_t key = 0;
    const float4 *quads = reinterpret_cast<const float4 *>(row + q0);
    int64_t q = tid;
    constexpr int kBatch = 8;  // loads in flight
    for (; q + (kBatch - 1) * kBestThreads < nq; q += kBatch * kBestThreads) {
        float4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) v[k] = __ldcs(quads + q + k * kBestThreads);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t i = static_cast<uint32_t>(q0 + 4 * (q + k * kBestThreads));
            key = max(key, max(max(best_key(v[k].x, i), best_key(v[k].y, i + 1)),
                               max(best_key(v[k].z, i + 2), best_key(v[k].w, i + 3))));
        }
    }
    for (; q < nq; q += kBestThreads) {
        const float4 v = __ldcs(quads + q);
        const uint32_t i = static_cast<uint32_t>(q0 + 4 * q);
        key = max(key, max(max(best_key(v.x, i), best_key(v.y, i + 1)), max(best_key(v.z, i + 2), best_key(v.w, i + 3))));
    }
    if (tid < q0 - lo) key = max(key, best_key(row[lo + tid], static_cast<uint32_t>(lo + tid)));
    const int64_t rest = q0 + 4 * nq + tid;
    if (rest < hi) key = max(key, best_key(row[rest], static_cast<uint32_t>(rest)));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
    if ((tid & 31) == 0) s_key[tid >> 5] = key;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kBestThreads / 32; ++w) key = max(key, s_key[w]);
        parts[blockIdx.x] = key;
    }
}

// A block a request, a warp a draft for the answers of its slices, then a thread
// a draft (block B: the padding rows).  The first right child of every draft is
// found by all threads at once; one thread then follows the chain.  2 us beside
// best_kernel's, with the early start.
__global__ void __launch_bounds__(ABG_MAX_SPAN) accept_kernel(const int32_t *tok, const int32_t *parent,
                                                              const int32_t *cu, int32_t *best, int32_t *rows,
                                                              int32_t *add, int32_t *last, int B, int N, int splits,
                                                              const uint64_t *parts) {
    __shared__ int s_best[ABG_MAX_SPAN], s_next[ABG_MAX_SPAN], s_path[ABG_MAX_SPAN], s_count;
    const int b = blockIdx.x, i = threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    const int lo = max(0, b < B ? cu[b] : cu[B]), hi = min(N, b < B ? cu[b + 1] : N);
    const int T = b < B ? max(0, min(hi - lo, ABG_MAX_SPAN)) : 0;
    for (int64_t n = static_cast<int64_t>(lo) + (i >> 5); n < hi; n += ABG_MAX_SPAN / 32) {
        uint64_t key = 0;
        for (int s = i & 31; s < splits; s += 32) key = max(key, parts[n * splits + s]);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
        if ((i & 31) == 0) {
            const int v = static_cast<int32_t>(~static_cast<uint32_t>(key));
            best[n] = v;
            rows[n] = -1;
            if (n - lo < T) s_best[n - lo] = v;
        }
    }
    if (b >= B) return;
    s_next[i] = ABG_MAX_SPAN;
    __syncthreads();
    if (i < T) {
        const int p = parent[lo + i];
        if (p >= 0 && p < i && tok[lo + i] == s_best[p]) atomicMin(&s_next[p], i);  // in shared memory
    }
    __syncthreads();
    if (i == 0) {
        int count = 0;
        for (int at = 0; at < T; at = s_next[at]) s_path[count++] = at;
        s_count = count;
        add[b] = count;
        last[b] = count ? s_best[s_path[count - 1]] : -1;
    }
    __syncthreads();
    if (i < s_count) rows[lo + i] = lo + s_path[i];
}

constexpr int64_t kSlice = 4096;  // shortest slice

int64_t best_slices(int64_t N, int64_t V) {
    // four blocks an SM, all at once (304 rows: 54.0 us; eight blocks 54.7)
    const int64_t want = std::max<int64_t>(1, 4 * sm_count() / std::max<int64_t>(1, N));
    return std::max<int64_t>(1, std::min<int64_t>(want, (V + kSlice - 1) / kSlice));
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs &a, bool pdl, cudaStream_t stream) {
    const size_t smem = (2 * static_cast<size_t>(a.B) + 1) * sizeof(int32_t);
    static const cudaError_t attr = cudaFuncSetAttribute(
        page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (2 * ABG_MAX_REQUESTS + 1) * sizeof(int32_t));
    if (attr != cudaSuccess) return attr;
    // four tokens a thread; a request a warp; one wave of two blocks an SM (a
    // second wave: 12.3 us against 10.3 for the 768000 tokens)
    const int64_t tokens = (a.N + 4ll * kPlanThreads - 1) / (4 * kPlanThreads);
    const int table_blocks = (32 * a.B + kPlanThreads - 1) / kPlanThreads;
    const int token_blocks = static_cast<int>(std::min<int64_t>(tokens, std::max(sm_count(), 2 * sm_count() - table_blocks)));
    // An early start deals blocks to the SMs that the launch ahead leaves first,
    // so that some get more than their share: for short grids only (384 tokens:
    // 8.2 us, early 5.2; 768000 tokens: 10.3 us, early 11.4 when one block did
    // both kinds of work, 9.9 with the tables on blocks of their own).
    const bool early = pdl && token_blocks + table_blocks <= sm_count() && !capturing(stream);
    return launch_kernel(page_plan_kernel, dim3(static_cast<unsigned>(token_blocks + table_blocks)), dim3(kPlanThreads),
                         smem, stream, early, a, token_blocks);
}

cudaError_t launch_tree_plan(const int32_t *parent, const int32_t *lens, const int32_t *cu, uint64_t *mask,
                             int32_t *pos, int B, int N, int words, bool pdl, cudaStream_t stream) {
    auto *fn = words == 1   ? tree_plan_kernel<1>
               : words == 2 ? tree_plan_kernel<2>
               : words == 3 ? tree_plan_kernel<3>
                            : tree_plan_kernel<4>;
    return launch_kernel(fn, dim3(static_cast<unsigned>(B) + 1), dim3(64 * words), 0, stream,
                         pdl && !capturing(stream), parent, lens, cu, mask, pos, B, N);
}

template <typename S, typename T, int D>
static cudaError_t put_d(const abg_kv_put_args &a, bool early, cudaStream_t stream) {
    // as many blocks as fit at once
    static const int fit = [] {
        int per = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kv_put_kernel<S, T, D>, 32 * kPutWarps, 0) !=
            cudaSuccess)
            per = 1;
        return std::max(per, 1) * sm_count();
    }();
    const int heads = static_cast<int>((a.q ? a.Hq : 0) + 2 * a.Hkv);
    const int groups = (heads + Put<D>::kHeads - 1) / Put<D>::kHeads;
    const int64_t blocks = (a.N * groups + kPutWarps - 1) / kPutWarps;
    return launch_kernel(kv_put_kernel<S, T, D>, dim3(static_cast<unsigned>(std::min<int64_t>(blocks, fit))),
                         dim3(32 * kPutWarps), 0, stream, early, a, groups);
}
template <typename S, typename T>
static cudaError_t put(const abg_kv_put_args &a, bool early, cudaStream_t stream) {
    return a.D == 64    ? put_d<S, T, 64>(a, early, stream)
           : a.D == 128 ? put_d<S, T, 128>(a, early, stream)
                        : put_d<S, T, 256>(a, early, stream);
}

cudaError_t launch_kv_put(const abg_kv_put_args &a, bool pdl, cudaStream_t stream) {
    const bool f32 = a.src_type == ABG_SB_F32, early = pdl && !capturing(stream);
    switch (a.type) {
    case ABG_SB_F32: return put<float, float>(a, early, stream);
    case ABG_SB_BF16:
        return f32 ? put<float, __nv_bfloat16>(a, early, stream) : put<__nv_bfloat16, __nv_bfloat16>(a, early, stream);
    default: return f32 ? put<float, __half>(a, early, stream) : put<__half, __half>(a, early, stream);
    }
}

size_t tree_accept_bytes(int64_t N, int64_t V) {
    return static_cast<size_t>(N * best_slices(N, V)) * sizeof(uint64_t);
}

cudaError_t launch_tree_accept(const float *logits, int64_t ld, const int32_t *tok, const int32_t *parent,
                               const int32_t *cu, int32_t *best, int32_t *rows, int32_t *add, int32_t *last, int B,
                               int N, int64_t V, void *ws, bool pdl, cudaStream_t stream) {
    const int64_t slices = best_slices(N, V);
    const int64_t slice = (V + slices - 1) / slices;
    uint64_t *parts = static_cast<uint64_t *>(ws);
    if (N > 0) {
        // early where there is not work for all SMs, as page_plan (304 rows: 54.0
        // us, early 59.0; eight rows: 8.2 us, early 6.4)
        const bool early = pdl && slices == (V + kSlice - 1) / kSlice && !capturing(stream);
        const cudaError_t e = launch_kernel(best_kernel, dim3(static_cast<unsigned>(slices * N)), dim3(kBestThreads), 0,
                                            stream, early, logits, ld, V, slices, slice, parts);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(accept_kernel, dim3(static_cast<unsigned>(B) + 1), dim3(ABG_MAX_SPAN), 0, stream, pdl && N > 0, tok,
                         parent, cu, best, rows, add, last, B, N, slices, parts);
}

}  // namespace abg
