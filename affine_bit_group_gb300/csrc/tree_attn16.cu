// tree_attn for 16-bit types on the tensor cores (formulas in include/abg.h,
// the work split in tree_attn.cuh).
//
// A block holds 128 query rows (drafts x heads of one key/value head) and
// streams token tiles past them, one pass with a running maximum:
//
//   S = Q K^T     tcgen05.mma, Q and K in shared memory, S (f32) in TMEM
//   P = 2^(S - m) four warps, a thread a row, from TMEM through registers back
//                 into TMEM as 16-bit values over S's own columns
//   O += P V      tcgen05.mma with P read from TMEM, V from shared memory
//
// Warps 0-3 are the softmax rows (TMEM lanes 32w ..), warp 4 brings K and V
// tiles with TMA into a ring of tile-sized slots, lane 0 of warp 5 issues the
// matrix instructions.  S has two buffers: the product of tile j+1 runs while
// the weights of tile j are taken.  The pages of the cache need not be aligned
// to tiles: a tile is copied in boxes of the largest power of two of rows that
// divides the page, each from its own page.
//
// Why 128 rows even for a few drafts: the matrix unit has 128 rows, and a tile's
// product with all of them takes 0.65 us of an SM's tensor time per 64 KB of
// cache, less than half of the 1.5 us its share of the memory bandwidth takes
// to deliver them.  Rows past the unit's are not loaded, and warps without rows
// skip the softmax.
#include "abg_kernels.cuh"
#include "tree_attn.cuh"
#include "tree_attn16.cuh"

#include <cuda.h>

#include <algorithm>
#include <cmath>

namespace abg {

namespace {

constexpr int kRT = 128;
constexpr int kThreads16 = 192;
constexpr int kDraftBox = 16;  // rows of a box of the draft buffers

template <int D>
struct Shape {
    static constexpr int kKT = D == 256 ? 64 : 128;      // tokens a tile
    static constexpr int kCols = D / 64;                  // 128-byte column blocks
    static constexpr uint32_t kQBytes = kRT * D * 2;
    static constexpr uint32_t kTile = kKT * D * 2;        // a K or V tile: a ring slot
    static constexpr int kSlots = D == 64 ? 12 : D == 128 ? 6 : 5;
    static constexpr uint32_t kSmem = 1024 + kQBytes + kSlots * kTile;
};
constexpr uint32_t kTmemO = 256;  // TMEM columns: S buffers at 0 and 128, O from 256 on

struct Maps {
    CUtensorMap k, v, kd, vd;
};

struct Bars {
    uint64_t full[12], empty[12];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t q_full, o_free, drain;
};

// ------------------------------------------------------------ PTX wrappers --
__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two values rounded to T, the first in the lower half
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t r;
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    } else {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    }
    return r;
}

// Shared-memory operand in 128-byte swizzle.  K-major (rows of 64 elements of
// the summed dimension): 8-row groups 1024 bytes apart.  MN-major (V: rows are
// the summed tokens): `lead` bytes between blocks of 64 columns, 8-token
// groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// f32 accumulator, A and B of type T, A K-major, B K-major or (b_mn) MN-major
template <typename T>
__host__ __device__ constexpr uint32_t instr_desc(int m, int n, bool b_mn) {
    const uint32_t t = std::is_same_v<T, __nv_bfloat16> ? 1 : 0;
    return 1u << 4 | t << 7 | t << 10 | (b_mn ? 1u << 16 : 0u) | static_cast<uint32_t>(n / 8) << 17 |
           static_cast<uint32_t>(m / 16) << 24;
}

// A wait that gives up after kWaitLimitNs, or at once when another thread of
// the block has: the kernel then drains its copies, frees its TMEM and ends,
// with the device status word set.
__device__ __forceinline__ bool wait16(uint64_t *bar, uint32_t parity, volatile int *gone) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
        if (*gone) return false;
        if (globaltimer() - t0 > kWaitLimitNs) {
            *gone = 1;
            atomicOr(&g_status, kStatusTimeout | (1u << 8));
            return false;
        }
    }
}

// Tokens of tile t of a stretch's unit, 1 .. kKT.
template <int kKT>
__device__ __forceinline__ int tile_tokens(const AttnSeg &s, int t) {
    return t < s.ctiles ? min(kKT, s.req.len - t * kKT) : min(kKT, s.req.T - (t - s.ctiles) * kKT);
}

// A place on the block's tile stream.
template <int kKT>
struct Cursor {
    AttnLine<kRT, kKT> line;
    AttnSeg s;
    int t;
    bool on;
    __device__ __forceinline__ void start(const AttnArgs &p, const AttnLine<kRT, kKT> &l) {
        line = l;
        on = line.next(p, s);
        t = s.t0;
    }
    __device__ __forceinline__ void step(const AttnArgs &p) {
        if (++t == s.t1) {
            on = line.next(p, s);
            t = s.t0;
        }
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads16, 1) attn16_kernel(const __grid_constant__ AttnArgs p,
                                                              const __grid_constant__ Maps maps, int box) {
    using S = Shape<D>;
    constexpr int kKT = S::kKT, kSlots = S::kSlots, kCols = S::kCols;
    extern __shared__ unsigned char raw[];
    __shared__ Bars bars;
    __shared__ uint32_t s_tmem;
    __shared__ uint32_t s_bad[2][ABG_MAX_SPAN / 32];
    __shared__ volatile int s_gone;
    const abg_tree_attn_args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned char *base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char *sm_q = base, *sm_ring = base + S::kQBytes;
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        s_gone = 0;
        for (int i = 0; i < kSlots; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < 2; ++i)
            mbar_init(&bars.s_full[i], 1), mbar_init(&bars.p_full[i], 4), mbar_init(&bars.pv_done[i], 1);
        mbar_init(&bars.q_full, 4), mbar_init(&bars.o_free, 4), mbar_init(&bars.drain, 1);
        fence_mbar_init();
    }
    tc_before();
    grid_dep_wait();
    grid_dep_launch();
    AttnLine<kRT, kKT> line;
    line.template init<kThreads16>(p, blockIdx.x, gridDim.x);
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    const int n_tiles = static_cast<int>(line.end - line.cur);
    // ring items: K0, then K(j+1), V(j) in turn
    auto item_k = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto item_v = [n_tiles](int j) { return j < n_tiles - 1 ? 2 * j + 2 : 2 * j + 1; };
    auto slot = [&](int i) { return sm_ring + static_cast<uint32_t>(i % kSlots) * S::kTile; };

    if (warp == 4) {
        // ------------------------------------------------- the copying warp
        Cursor<kKT> ck, cv;
        ck.start(p, line);
        cv.start(p, line);
        int items = 0;
        bool live = true;
        auto bring = [&](const Cursor<kKT> &c, bool value) {
            const AttnSeg &s = c.s;
            const bool cache = c.t < s.ctiles;
            const int step = cache ? box : kDraftBox;
            const int boxes = (tile_tokens<kKT>(s, c.t) + step - 1) / step;
            const CUtensorMap *map = cache ? (value ? &maps.v : &maps.k) : (value ? &maps.vd : &maps.kd);
            unsigned char *to = slot(items);
            uint64_t *bar = &bars.full[items % kSlots];
            const int key0 = c.t * kKT, page = static_cast<int>(a.page);
            // where the lane's first box lies (the load is in flight during the wait)
            auto where = [&](int i, int &y, int &z) {
                if (cache) {
                    const int key = key0 + i * step, j = key / page;
                    const int64_t id = a.table[static_cast<int64_t>(s.b) * a.width + j];
                    y = key - j * page;
                    z = id >= 0 && id < a.pages ? static_cast<int>(id * a.Hkv) + s.h : -1;  // -1: zeros
                } else {
                    y = s.req.n0 + (c.t - s.ctiles) * kKT + i * step;
                    z = s.h;
                }
            };
            int y = 0, z = 0;
            if (lane < boxes) where(lane, y, z);
            if (items >= kSlots && live) live = wait16(&bars.empty[items % kSlots], (items / kSlots - 1) & 1, &s_gone);
            live = __all_sync(0xffffffffu, live);
            if (!live) return;
            if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * step) * D * 2);
            __syncwarp();
            for (int i = lane; i < boxes; i += 32) {
                if (i != lane) where(i, y, z);
#pragma unroll
                for (int cb = 0; cb < kCols; ++cb)
                    tma_3d(to + static_cast<uint32_t>(cb) * kKT * 128 + static_cast<uint32_t>(i * step) * 128, map,
                           64 * cb, y, z, bar);
            }
            ++items;
        };
        if (n_tiles > 0) {
            bring(ck, false);
            for (int j = 0; j < n_tiles && live; ++j) {
                if (j + 1 < n_tiles) {
                    ck.step(p);
                    bring(ck, false);
                }
                if (live) bring(cv, true);
                cv.step(p);
            }
        }
        if (!live)  // what was issued must have landed before the block ends
            for (int i = max(0, items - kSlots); i < items; ++i) mbar_wait(&bars.full[i % kSlots], (i / kSlots) & 1);
    } else if (warp == 5) {
        // --------------------------------------------- the issuing thread
        if (lane == 0 && n_tiles > 0) {
            constexpr uint32_t kQK = instr_desc<T>(kRT, kKT, false), kPV = instr_desc<T>(kRT, D, true);
            const uint32_t q = smem_u32(sm_q);
            int seg = 0;
            bool live = true;
            auto product = [&](int j) {  // S(j) = Q K(j)^T
                const int i = item_k(j);
                live = live && wait16(&bars.full[i % kSlots], (i / kSlots) & 1, &s_gone) &&
                       (j < 2 || wait16(&bars.pv_done[j & 1], ((j - 2) >> 1) & 1, &s_gone));
                if (!live) return;
                tc_after();
                const uint32_t k = smem_u32(slot(i));
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
                    mma_ss(tmem + (j & 1) * 128, smem_desc(q + (d / 4) * (kRT * 128) + (d % 4) * 32, 16),
                           smem_desc(k + (d / 4) * (kKT * 128) + (d % 4) * 32, 16), kQK, d > 0);
                tc_commit(&bars.s_full[j & 1]);
                tc_commit(&bars.empty[i % kSlots]);
            };
            AttnSeg s;
            for (int j = 0; live && line.next(p, s); ++seg) {
                live = wait16(&bars.q_full, seg & 1, &s_gone);
                product(j);
                for (int t = s.t0; live && t < s.t1; ++t, ++j) {
                    if (t + 1 < s.t1) product(j + 1);  // ahead of this tile's sums
                    const int i = item_v(j);
                    live = live && wait16(&bars.full[i % kSlots], (i / kSlots) & 1, &s_gone) &&
                           wait16(&bars.p_full[j & 1], (j >> 1) & 1, &s_gone) &&
                           (t > s.t0 || seg == 0 || wait16(&bars.o_free, (seg - 1) & 1, &s_gone));
                    if (!live) break;
                    tc_after();
                    const uint32_t v = smem_u32(slot(i));
                    const int steps = (tile_tokens<kKT>(s, t) + 15) / 16;  // past the tokens there is no weight
                    for (int k = 0; k < steps; ++k)
                        mma_ts(tmem + kTmemO, tmem + (j & 1) * 128 + k * 8, smem_desc(v + k * 2048, kKT * 128), kPV,
                               t > s.t0 || k > 0);
                    tc_commit(&bars.pv_done[j & 1]);
                    tc_commit(&bars.empty[i % kSlots]);
                }
            }
            if (!live) {  // matrix instructions in flight read this block's memory
                tc_commit(&bars.drain);
                mbar_wait(&bars.drain, 0);
            }
        }
    } else {
        // ------------------------------------------------ the softmax rows
        AttnSplit split{};
        AttnSeg s;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const int r = tid;  // row of the tile
        bool live = true;
        int j = 0, seg = 0;
        for (; live && line.next(p, s); ++seg) {
            const bool busy = warp * 32 < s.rows, mine = r < s.rows;
            uint32_t *bad = s_bad[seg & 1];
            if (tid < ABG_MAX_SPAN / 32) bad[tid] = 0;
            // Q, swizzled: 16-byte chunk ch of row q at chunk ch ^ (q % 8).  The
            // products that read the last stretch's Q are done (their S was).
            for (int i = tid; i < s.rows * (D / 8); i += 128) {
                const int q = i / (D / 8), ch = i % (D / 8), row = s.r0 + q;
                const uint4 v = *reinterpret_cast<const uint4 *>(
                    static_cast<const T *>(a.q) +
                    ((static_cast<int64_t>(s.req.n0) + row / p.G) * a.Hq + s.h * p.G + row % p.G) * D + ch * 8);
                *reinterpret_cast<uint4 *>(sm_q + (ch / 8) * (kRT * 128) + q * 128 + ((ch % 8) ^ (q % 8)) * 16) = v;
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.q_full);
            const int64_t n = static_cast<int64_t>(s.req.n0) + (s.r0 + (mine ? r : 0)) / p.G;
            const uint64_t *seen = a.mask + n * a.words;
            float ref = -INFINITY, l = 0.0f;
            for (int t = s.t0; t < s.t1; ++t, ++j) {
                const bool drafts = t >= s.ctiles;
                const int tokens = tile_tokens<kKT>(s, t), key0 = (t - s.ctiles) * kKT;
                const uint32_t sbuf = tmem + (j & 1) * 128 + lanes;
                live = wait16(&bars.s_full[j & 1], (j >> 1) & 1, &s_gone);
                live = __all_sync(0xffffffffu, live);
                if (!live) break;
                tc_after();
                if (busy) {
                    float x[kKT];
#pragma unroll
                    for (int k = 0; k < kKT; k += 32) tmem_ld32(sbuf + k, *reinterpret_cast<float(*)[32]>(x + k));
                    tmem_ld_wait();
                    if (drafts) {
#pragma unroll
                        for (int w = 0; w < kKT / 64; ++w) {
                            uint64_t bits = key0 / 64 + w < a.words ? seen[key0 / 64 + w] : 0;
                            const int left = tokens - 64 * w;
                            if (left < 64) bits &= left > 0 ? (1ull << left) - 1 : 0;
#pragma unroll
                            for (int k = 0; k < 64; ++k)
                                if (!(bits >> k & 1)) x[64 * w + k] = -INFINITY;
                        }
                    } else if (tokens < kKT) {
#pragma unroll
                        for (int k = 0; k < kKT; ++k)
                            if (k >= tokens) x[k] = -INFINITY;
                    }
                    float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int k = 4; k < kKT; ++k) top[k & 3] = fmaxf(top[k & 3], x[k]);
                    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale2;
                    // The reference follows the maximum only when it is 2^8
                    // behind: weights up to 256 lose nothing in 16 bits, and
                    // rescaling O costs a round trip through TMEM.
                    const bool up = mx > ref + 8.0f;
                    if (__any_sync(0xffffffffu, up)) {
                        const float to = up ? mx : ref;
                        const float f = up ? ex2(ref - to) : 1.0f;
                        ref = to;
                        l *= f;
                        if (t > s.t0) {
                            live = wait16(&bars.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, &s_gone);
                            live = __all_sync(0xffffffffu, live);
                            if (!live) break;
                            tc_after();
#pragma unroll 1
                            for (int k = 0; k < D; k += 32) {
                                float o[32];
                                tmem_ld32(tmem + kTmemO + lanes + k, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= f;
                                tmem_st32(tmem + kTmemO + lanes + k, *reinterpret_cast<uint32_t(*)[32]>(o));
                            }
                        }
                    }
                    const float sub = ref == -INFINITY ? 0.0f : ref;
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < kKT; k += 64) {
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float e0 = ex2(fmaf(x[k + 2 * i], p.scale2, -sub));
                            const float e1 = ex2(fmaf(x[k + 2 * i + 1], p.scale2, -sub));
                            sum[(2 * i) & 3] += e0;
                            sum[(2 * i + 1) & 3] += e1;
                            w[i] = pack2<T>(e0, e1);
                        }
                        tmem_st32(sbuf + k / 2, w);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_st_wait();
                }
                if (drafts || tokens < kKT) {
                    // V rows past the tile's tokens hold what was there before,
                    // and a draft's V may hold an infinity or a NaN that only
                    // the rows that see it may get: 0 * NaN is NaN, so both are
                    // cleared here (the latter is added back at the end).
                    const int i = item_v(j), all = (tokens + 15) / 16 * 16;
                    live = wait16(&bars.full[i % kSlots], (i / kSlots) & 1, &s_gone);
                    live = __all_sync(0xffffffffu, live);
                    if (!live) break;
                    unsigned char *v = slot(i);
                    for (int e = tid; e < all * (D / 8); e += 128) {
                        const int row = e / (D / 8), ch = e % (D / 8);
                        uint4 *at = reinterpret_cast<uint4 *>(v + (ch / 8) * (kKT * 128) + row * 128 +
                                                              ((ch % 8) ^ (row % 8)) * 16);
                        if (row >= tokens) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else if (drafts) {
                            constexpr uint32_t kExp = std::is_same_v<T, __nv_bfloat16> ? 0x7f80u : 0x7c00u;
                            uint4 u = *at;
                            uint32_t *h = reinterpret_cast<uint32_t *>(&u);
                            bool hit = false;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if ((h[q] & kExp) == kExp) h[q] &= 0xffff0000u, hit = true;
                                if ((h[q] >> 16 & kExp) == kExp) h[q] &= 0xffffu, hit = true;
                            }
                            if (hit) {
                                *at = u;
                                atomicOr(&bad[(key0 + row) >> 5], 1u << ((key0 + row) & 31));
                            }
                        }
                    }
                    fence_async();
                }
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[j & 1]);
            }
            if (!live) break;
            // the stretch's sums: tile j-1 was its last
            live = wait16(&bars.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, &s_gone);
            live = __all_sync(0xffffffffu, live);
            if (!live) break;
            tc_after();
            const bool whole = s.t0 == 0 && s.t1 == s.tiles;
            const int64_t piece = (static_cast<int64_t>(2) * blockIdx.x + (s.t0 == 0)) * kRT + r;
            const int64_t at = (n * a.Hq + s.h * p.G + (s.r0 + (mine ? r : 0)) % p.G) * D;
            if (busy) {
                float group = 0.0f;
                const float scale = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    __syncwarp();  // rows past the unit's have skipped ahead
                    tmem_ld32(tmem + kTmemO + lanes + k, o);
                    tmem_ld_wait();
                    if (!mine) continue;
                    for (int w = 0; w < (s.req.T + 31) / 32; ++w)
                        for (uint32_t m = bad[w]; m; m &= m - 1) {
                            const int d = 32 * w + __ffs(static_cast<int>(m)) - 1;
                            if (!attn_sees(seen, d)) continue;
                            const T *vd = static_cast<const T *>(a.Vd) +
                                          (s.h * a.drafts + s.req.n0 + d) * static_cast<int64_t>(D) + k;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float v = static_cast<float>(vd[i]);
                                if (!(fabsf(v) < INFINITY)) o[i] += v;
                            }
                        }
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(p.part_o + piece * D + k + i) =
                                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = l == 0.0f ? 0.0f : o[i] * scale;
                    if (a.gate)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 g = *reinterpret_cast<const float4 *>(a.gate + at + k + i);
                            o[i] /= 1.0f + __expf(-g.x), o[i + 1] /= 1.0f + __expf(-g.y);
                            o[i + 2] /= 1.0f + __expf(-g.z), o[i + 3] /= 1.0f + __expf(-g.w);
                        }
                    if (a.y_type == ABG_SB_F32) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(static_cast<float *>(a.y) + at + k + i) =
                                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + at + k + i) =
                                make_uint4(pack2<T>(o[i], o[i + 1]), pack2<T>(o[i + 2], o[i + 3]),
                                           pack2<T>(o[i + 4], o[i + 5]), pack2<T>(o[i + 6], o[i + 7]));
                    }
                    if (a.ysum) {
                        float sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum += o[i];
                        group += sum;
                        if (k & 32) a.ysum[(at + k) / 64] = group, group = 0.0f;
                    }
                }
                if (mine && !whole) p.part_ml[piece] = make_float2(ref, l);
            }
            if (s.t0 == 0 && s.t1 < s.tiles)
                split = AttnSplit{s.req.n0, s.h, s.r0, s.rows, line.block_of_end(s.unit + s.tiles)};
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.o_free);
        }
        if (tid == 0) p.split[blockIdx.x] = split;
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 5)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ------------------------------------------------------------------ host ---
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &res) !=
                cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// Rows of D 16-bit values as [outer][rows][D], copied in boxes of box x 64.
template <typename T>
bool row_map(CUtensorMap *map, const void *p, int64_t D, int64_t rows, int64_t outer, int box) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(rows * D) * 2};
    const cuuint32_t tile[3] = {64, static_cast<cuuint32_t>(box), 1}, one[3] = {1, 1, 1};
    return encoder()(map,
                     std::is_same_v<T, __nv_bfloat16> ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     3, const_cast<void *>(p), dims, strides, tile, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t go16(AttnArgs p, void *ws, cudaStream_t stream) {
    using S = Shape<D>;
    static const cudaError_t attr =
        cudaFuncSetAttribute(attn16_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (attr != cudaSuccess) return attr;
    if (!encoder()) return cudaErrorSymbolNotFound;
    const abg_tree_attn_args &a = p.a;
    // a box lies in one page: the largest power of two of rows that divides it
    const int box = static_cast<int>(std::min<int64_t>(a.page & -a.page, S::kKT));
    const bool cached = a.pages > 0 && a.width > 0;
    Maps m;
    if (!row_map<T>(&m.k, cached ? a.Kc : a.Kd, D, cached ? a.page : a.drafts, cached ? a.pages * a.Hkv : a.Hkv, box) ||
        !row_map<T>(&m.v, cached ? a.Vc : a.Vd, D, cached ? a.page : a.drafts, cached ? a.pages * a.Hkv : a.Hkv, box) ||
        !row_map<T>(&m.kd, a.Kd, D, a.drafts, a.Hkv, kDraftBox) ||
        !row_map<T>(&m.vd, a.Vd, D, a.drafts, a.Hkv, kDraftBox))
        return cudaErrorInvalidValue;
    const int C = sm_count();
    const AttnLayout l = attn_layout(C, kRT, D);
    unsigned char *w = static_cast<unsigned char *>(ws);
    p.part_o = reinterpret_cast<float *>(w + l.o);
    p.part_ml = reinterpret_cast<float2 *>(w + l.ml);
    p.split = reinterpret_cast<AttnSplit *>(w + l.split);
    const cudaError_t e =
        launch_kernel(attn16_kernel<T, D>, dim3(C), dim3(kThreads16), S::kSmem, stream, false, p, m, box);
    if (e != cudaSuccess) return e;
    return launch_kernel(attn_join_kernel<T, D, kRT>, dim3(C, kRT / 8), dim3(256), 0, stream, true, p);
}

}  // namespace

size_t tree_attn16_bytes(int D) { return attn_layout(sm_count(), kRT, D).total; }

cudaError_t launch_tree_attn16(const AttnArgs &p, void *ws, cudaStream_t stream) {
    const bool bf = p.a.type == ABG_SB_BF16;
    switch (p.a.D) {
    case 64: return bf ? go16<__nv_bfloat16, 64>(p, ws, stream) : go16<__half, 64>(p, ws, stream);
    case 128: return bf ? go16<__nv_bfloat16, 128>(p, ws, stream) : go16<__half, 128>(p, ws, stream);
    default: return bf ? go16<__nv_bfloat16, 256>(p, ws, stream) : go16<__half, 256>(p, ws, stream);
    }
}

// This unit's device status word (OR-ed into *bits).
cudaError_t tree_attn16_status(unsigned *bits, bool clear) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof v);
    if (e == cudaSuccess && clear && v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_status, &zero, sizeof zero);
    }
    *bits |= v;
    return e;
}

}  // namespace abg
