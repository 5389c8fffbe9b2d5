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
// that no block waits for another; the blocks then share the tokens.  A token
// of a fresh page takes the page from the ring itself, not from the table
// entry that another block writes.
constexpr int kPlanThreads = 512;

__device__ __forceinline__ int ring_at(int64_t i, int len) {
    const int r = static_cast<int>(i % len);
    return r < 0 ? r + len : r;
}

struct Ask {
    int64_t total, need;
    bool gone, bad;
    int64_t extra, freed;
};

__device__ __forceinline__ Ask ask_of(const PagePlanArgs &a, int b) {
    Ask k;
    const int64_t len = a.lens[b], add = a.add[b], held = a.held[b];
    const int64_t span = static_cast<int64_t>(a.cu[b + 1]) - a.cu[b];
    k.gone = add < 0;
    k.total = len + add;
    k.need = (k.total + a.page - 1) / a.page;
    k.bad = len < 0 || held < 0 || held > a.width ||
            (!k.gone && (add > span || k.need > a.width || k.total > 0x7fffffff));
    k.extra = k.gone || k.bad ? 0 : max(int64_t(0), k.need - held);
    k.freed = k.gone && !k.bad ? held : 0;
    return k;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PagePlanArgs a) {
    extern __shared__ int32_t sm[];
    int32_t *s_cu = sm;              // [B+1]
    int32_t *s_at = sm + a.B + 1;    // [B] ring entry of the first fresh or freed page; -1: refused
    __shared__ int64_t s_sum[2][kPlanThreads / 32];
    __shared__ int s_bad[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_wait();
    const int64_t head = a.ends[0], tail = a.ends[1];
    const int64_t avail = max(int64_t(0), min(tail - head, static_cast<int64_t>(a.ring_len)));
    int64_t done_x = 0, done_f = 0, taken = 0;  // taken: extras up to the last request that was granted any
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
            const bool done = k.gone && !k.bad;
            if (ok && k.extra > 0) taken = x;
            bad += !ok && !done;
            s_at[b] = ok     ? ring_at(head + x - k.extra, a.ring_len)
                      : done ? ring_at(tail + f - k.freed, a.ring_len)
                             : -1;
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
            bad += __shfl_xor_sync(0xffffffffu, bad, d);
        }
        if (lane == 0) s_sum[0][warp] = taken, s_bad[warp] = bad;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        for (int w = 1; w < kPlanThreads / 32; ++w) taken = max(taken, s_sum[0][w]), bad += s_bad[w];
        a.ends_out[0] = head + taken;
        a.ends_out[1] = tail + done_f;
        a.info[0] = static_cast<int32_t>(taken);
        a.info[1] = bad;
    }
    // table and ring entries: a warp a request
    const int gw = blockIdx.x * (kPlanThreads / 32) + warp, nw = gridDim.x * (kPlanThreads / 32);
    for (int b = gw; b < a.B; b += nw) {
        const int at = s_at[b];
        if (at < 0) continue;
        int32_t *row = a.table + static_cast<int64_t>(b) * a.width;
        const Ask k = ask_of(a, b);
        const int held = a.held[b];
        for (int64_t j = lane; j < k.extra; j += 32) row[held + j] = a.ring[(at + j) % a.ring_len];
        for (int64_t j = lane; j < k.freed; j += 32) a.ring[(at + j) % a.ring_len] = row[j];
    }
    // slots: a thread a token
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid; n < a.N;
         n += static_cast<int64_t>(gridDim.x) * kPlanThreads) {
        int64_t slot = -1;
        int32_t pos = 0;
        const int b = request_of(s_cu, a.B, static_cast<int>(n));
        const int i = static_cast<int>(n) - s_cu[b], at = s_at[b];
        if (n < s_cu[a.B] && i >= 0 && at >= 0 && i < a.add[b]) {
            pos = a.lens[b] + i;
            const int j = pos / a.page, held = a.held[b];
            const int32_t id = j < held ? a.table[static_cast<int64_t>(b) * a.width + j]
                                        : a.ring[(static_cast<int64_t>(at) + j - held) % a.ring_len];
            slot = static_cast<int64_t>(id) * a.page + (pos - j * a.page);
        }
        a.slots[n] = slot;
        a.pos[n] = pos;
    }
}

// ---------------------------------------------------------- tree_plan ------
// A block a request, a thread a draft.  Each round a draft joins its pointer's
// mask to its own and moves the pointer to the pointer's pointer, so the
// pointer is 2^r ancestors away after r rounds: log2(span) rounds instead of
// the span's longest chain.  A cycle only repeats bits.
template <int W>
__global__ void __launch_bounds__(64 * W) tree_plan_kernel(const int32_t *parent, const int32_t *lens,
                                                           const int32_t *cu, uint64_t *mask, int32_t *pos, int B,
                                                           int N) {
    __shared__ uint64_t s_mask[2][W][64 * W];
    __shared__ int16_t s_up[2][64 * W];
    const int b = blockIdx.x, i = threadIdx.x;
    grid_dep_wait();
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
// A warp a token and four of its heads (q heads, then k, then v): lane l holds
// D/32 consecutive columns, so the squares are summed as the pairwise tree (the
// lane's values, then the butterfly) and column i + D/2 is in lane l ^ 16.
// The four heads' loads are issued before the first is used, and the token's
// rotation is read once for them.
constexpr int kPutHeads = 4;
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

template <typename S, typename T, int D>
__global__ void __launch_bounds__(32 * kPutWarps) kv_put_kernel(const __grid_constant__ abg_kv_put_args a,
                                                                int groups) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kPutWarps + (threadIdx.x >> 5);
    const int64_t n = unit / groups;
    const int h0 = static_cast<int>(unit - n * groups) * kPutHeads;
    grid_dep_wait();
    if (n >= a.N) return;
    const int64_t src = a.rows ? a.rows[n] : n;
    if (src < 0 || src >= a.src_rows) return;
    const int nq = a.q ? static_cast<int>(a.Hq) : 0, nk = static_cast<int>(a.Hkv);
    const int64_t slot = a.slots ? a.slots[n] : n;
    const bool kept = slot >= 0 && slot < a.pages * a.page;
    float u[kPutHeads][E];
    bool act[kPutHeads];
#pragma unroll
    for (int r = 0; r < kPutHeads; ++r) {
        const int h = h0 + r;
        act[r] = h < nq || (kept && h < nq + 2 * nk);
        if (!act[r]) continue;
        const S *p = h < nq        ? static_cast<const S *>(a.q) + src * a.q_row + h * a.q_head
                     : h < nq + nk ? static_cast<const S *>(a.k) + src * a.k_row + (h - nq) * a.k_head
                                   : static_cast<const S *>(a.v) + src * a.v_row + (h - nq - nk) * a.v_head;
        load_e<S, E>(p + lane * E, u[r]);
    }
    float c[E], s[E];
    if (a.cos) {
        const int32_t p = a.pos[n];
        const bool in = p >= 0 && p < a.cos_rows;
        const int64_t at = (in ? p : 0) * static_cast<int64_t>(D / 2) + (lane & 15) * E;
        load_e<float, E>(a.cos + at, c);
        load_e<float, E>(a.sin + at, s);
        if (!in)
#pragma unroll
            for (int i = 0; i < E; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
    }
    const int64_t page = kept ? slot / a.page : 0;
    const int64_t base = page * a.Hkv * a.page + (slot - page * a.page);
#pragma unroll
    for (int r = 0; r < kPutHeads; ++r) {
        const int h = h0 + r;
        if (!act[r]) continue;
        if (h < nq + nk) {
            const float *w = h < nq ? a.qn_w : a.kn_w;
            if (w) {
                float wv[E], t[E];
                load_e<float, E>(w + lane * E, wv);
#pragma unroll
                for (int i = 0; i < E; ++i) t[i] = __fmul_rn(u[r][i], u[r][i]);
#pragma unroll
                for (int k = E / 2; k >= 1; k >>= 1)
#pragma unroll
                    for (int i = 0; i < k; ++i) t[i] = __fadd_rn(t[2 * i], t[2 * i + 1]);
                const float ss = warp_tree<32>(t[0]);
                const float f = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(D)), a.eps)));
#pragma unroll
                for (int i = 0; i < E; ++i) u[r][i] = __fmul_rn(__fmul_rn(u[r][i], f), wv[i]);
            }
            if (a.cos) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float o = __shfl_xor_sync(0xffffffffu, u[r][i], 16);
                    const float uc = __fmul_rn(u[r][i], c[i]), os = __fmul_rn(o, s[i]);
                    u[r][i] = lane < 16 ? __fsub_rn(uc, os) : __fadd_rn(uc, os);
                }
            }
        }
        T *to = h < nq        ? static_cast<T *>(a.qo) + (n * a.Hq + h) * D
                : h < nq + nk ? static_cast<T *>(a.Kc) + (base + (h - nq) * a.page) * D
                              : static_cast<T *>(a.Vc) + (base + (h - nq - nk) * a.page) * D;
        store_e<T, E>(to + lane * E, u[r]);
    }
}

// --------------------------------------------------------- tree_accept -----
// The logits are read once, a block a slice of a row; a slice's answer is one
// 64-bit key, the value's order in the upper half and ~index in the lower, so
// that the largest key is the largest value at its lowest index.
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
    const int64_t lo = (blockIdx.x - n * slices) * slice, hi = min(V, lo + slice);
    // whole 16-byte quads from the first aligned element on, single ones around them
    const int64_t off = ((16 - (reinterpret_cast<uintptr_t>(row + lo) & 15)) & 15) / 4;
    const int64_t q0 = min(hi, lo + off), nq = (hi - q0) / 4;
    uint64_t key = 0;
    const float4 *quads = reinterpret_cast<const float4 *>(row + q0);
    int64_t q = tid;
    for (; q + 3 * kBestThreads < nq; q += 4 * kBestThreads) {
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __ldcs(quads + q + k * kBestThreads);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
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
    grid_dep_launch();
}

// A block a request, a thread a draft (block B: the padding rows).  The first
// right child of every draft is found by all threads at once; one thread then
// follows the chain.
__global__ void __launch_bounds__(ABG_MAX_SPAN) accept_kernel(const int32_t *tok, const int32_t *parent,
                                                              const int32_t *cu, int32_t *best, int32_t *rows,
                                                              int32_t *add, int32_t *last, int B, int N, int splits,
                                                              const uint64_t *parts) {
    __shared__ int s_best[ABG_MAX_SPAN], s_next[ABG_MAX_SPAN], s_path[ABG_MAX_SPAN], s_count;
    const int b = blockIdx.x, i = threadIdx.x;
    grid_dep_wait();
    const int lo = max(0, b < B ? cu[b] : cu[B]), hi = min(N, b < B ? cu[b + 1] : N);
    const int T = b < B ? max(0, min(hi - lo, ABG_MAX_SPAN)) : 0;
    for (int64_t n = static_cast<int64_t>(lo) + i; n < hi; n += ABG_MAX_SPAN) {
        uint64_t key = 0;
        for (int s = 0; s < splits; ++s) key = max(key, parts[n * splits + s]);
        best[n] = static_cast<int32_t>(~static_cast<uint32_t>(key));
        rows[n] = -1;
        if (n - lo < T) s_best[n - lo] = best[n];
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

int64_t best_slices(int64_t N, int64_t V) {
    // about four blocks an SM, slices of 4096 logits at least
    const int64_t want = std::max<int64_t>(1, 4 * 152 / std::max<int64_t>(1, N));
    return std::max<int64_t>(1, std::min<int64_t>(want, (V + 4095) / 4096));
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t stream) {
    const size_t smem = (2 * static_cast<size_t>(a.B) + 1) * sizeof(int32_t);
    static const cudaError_t attr = cudaFuncSetAttribute(
        page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (2 * ABG_MAX_REQUESTS + 1) * sizeof(int32_t));
    if (attr != cudaSuccess) return attr;
    const int64_t blocks = std::max<int64_t>((a.N + 4ll * kPlanThreads - 1) / (4 * kPlanThreads), (a.B + 63) / 64);
    return launch_kernel(page_plan_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 2 * sm_count()))),
                         dim3(kPlanThreads), smem, stream, false, a);
}

cudaError_t launch_tree_plan(const int32_t *parent, const int32_t *lens, const int32_t *cu, uint64_t *mask,
                             int32_t *pos, int B, int N, int words, cudaStream_t stream) {
    auto *fn = words == 1   ? tree_plan_kernel<1>
               : words == 2 ? tree_plan_kernel<2>
               : words == 3 ? tree_plan_kernel<3>
                            : tree_plan_kernel<4>;
    return launch_kernel(fn, dim3(static_cast<unsigned>(B) + 1), dim3(64 * words), 0, stream, false, parent, lens, cu,
                         mask, pos, B, N);
}

template <typename S, typename T>
static cudaError_t put_d(const abg_kv_put_args &a, dim3 grid, int groups, cudaStream_t stream) {
    auto *fn = a.D == 64 ? kv_put_kernel<S, T, 64> : a.D == 128 ? kv_put_kernel<S, T, 128> : kv_put_kernel<S, T, 256>;
    return launch_kernel(fn, grid, dim3(32 * kPutWarps), 0, stream, false, a, groups);
}

cudaError_t launch_kv_put(const abg_kv_put_args &a, cudaStream_t stream) {
    const int heads = static_cast<int>((a.q ? a.Hq : 0) + 2 * a.Hkv);
    const int groups = (heads + kPutHeads - 1) / kPutHeads;
    const int64_t blocks = (a.N * groups + kPutWarps - 1) / kPutWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
    const bool f32 = a.src_type == ABG_SB_F32;
    switch (a.type) {
    case ABG_SB_F32: return put_d<float, float>(a, grid, groups, stream);
    case ABG_SB_BF16:
        return f32 ? put_d<float, __nv_bfloat16>(a, grid, groups, stream)
                   : put_d<__nv_bfloat16, __nv_bfloat16>(a, grid, groups, stream);
    default:
        return f32 ? put_d<float, __half>(a, grid, groups, stream) : put_d<__half, __half>(a, grid, groups, stream);
    }
}

size_t tree_accept_bytes(int64_t N, int64_t V) {
    return static_cast<size_t>(N * best_slices(N, V)) * sizeof(uint64_t);
}

cudaError_t launch_tree_accept(const float *logits, int64_t ld, const int32_t *tok, const int32_t *parent,
                               const int32_t *cu, int32_t *best, int32_t *rows, int32_t *add, int32_t *last, int B,
                               int N, int64_t V, void *ws, cudaStream_t stream) {
    const int64_t slices = best_slices(N, V);
    const int64_t slice = (V + slices - 1) / slices;
    uint64_t *parts = static_cast<uint64_t *>(ws);
    if (N > 0) {
        const cudaError_t e = launch_kernel(best_kernel, dim3(static_cast<unsigned>(slices * N)), dim3(kBestThreads), 0,
                                            stream, false, logits, ld, V, slices, slice, parts);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(accept_kernel, dim3(static_cast<unsigned>(B) + 1), dim3(ABG_MAX_SPAN), 0, stream, N > 0, tok,
                         parent, cu, best, rows, add, last, B, N, slices, parts);
}

}  // namespace abg
