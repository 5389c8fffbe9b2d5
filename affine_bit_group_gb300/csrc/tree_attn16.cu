// tree_attn for 16-bit types on the tensor cores (formulas in include/abg.h,
// the work split in tree_attn.cuh).
//
// A block streams a unit's token tiles past its query rows (drafts x heads of
// one key/value head), one pass with a running maximum.  A step is
//
//   S = Q K^T     tcgen05.mma, Q and K in shared memory, S (f32) in TMEM
//   P = 2^(S - m) a warpgroup, a thread a row, from TMEM through registers back
//                 into TMEM as 16-bit values over S's own columns
//   O += P V      tcgen05.mma with P read from TMEM, V from shared memory
//
// for 128 rows and one tile, S in two buffers of TMEM.  With more than 128 rows in
// the unit two warpgroups have 128 of them each and take turns, one's
// exponentials beside the other's products, and each tile is read once for 256
// rows.  With fewer rows both take every tile, one its first 64 tokens and the
// other the rest, each with a maximum, a weight sum and an O of its own, joined
// at the end (a step's length is what bounds it there, and this halves its
// longest part; taking turns by tile measured 2850 cycles a tile against a
// memory share of 2800).  256 columns a head leave TMEM for one O only: there one
// warpgroup takes every step.
//
// Three warps (two, with one group) bring K and V tiles with TMA into a ring of
// tile-sized slots, one issues the matrix instructions.  The pages of the cache need not be aligned
// to tiles: a tile is copied in boxes of the largest power of two of rows that
// divides the page, each from its own page.
//
// Why 128 rows a step even for a few drafts: the matrix unit has 128 rows, and a
// tile's products with all of them take 0.65 us of an SM's tensor time per 64 KB
// of cache, less than half of the 1.5 us its share of the memory bandwidth takes
// to deliver them.  Rows past the unit's are not loaded, and warps without rows
// skip the softmax.
//
// Measured: 24 bf16 drafts on 32 ragged requests of 12000 tokens, 592 MB, 108.8 us
// with the joining (5.4 TB/s, 80% of a plain copy's rate; bytes bound it); 63 f16
// drafts on 131071 tokens of one request, 134 MB and 67.6 GFLOP, 76.8 us (0.88
// PFLOP/s; the chain product, softmax, product of one row group bounds it).  A box
// costs its warp about 130 cycles, so pages whose largest power of two is small
// are bound by their boxes: 8 bf16 drafts on 32 ragged requests of 6000 tokens, 128
// columns, in pages of 16, 24 or 128 tokens 62-63 us, of 100 (boxes of 4) 70, of 101
// (boxes of 1) 197.
#include "abg_kernels.cuh"
#include "tree_attn.cuh"
#include "tree_attn16.cuh"

#include <cuda.h>

#include <algorithm>
#include <cmath>

namespace abg {

namespace {

constexpr int kDraftBox = 16;  // rows of a box of the draft buffers

template <int D>
struct Shape {
    static constexpr int kGroups = D == 256 ? 1 : 2;      // warpgroups of rows
    static constexpr int kRT = 128 * kGroups;             // rows of a unit
    static constexpr int kCopyWarps = kGroups == 2 ? 3 : 2;
    static constexpr int kThreads = 128 * kGroups + 32 * (1 + kCopyWarps);
    static constexpr int kKT = D == 256 ? 64 : 128;       // tokens a tile
    static constexpr int kCols = D / 64;                  // 128-byte column blocks
    static constexpr uint32_t kQTile = 128 * D * 2;
    static constexpr uint32_t kQBytes = kQTile * kGroups;
    static constexpr uint32_t kTile = kKT * D * 2;        // a K or V tile: a ring slot
    static constexpr int kSlots = D == 64 ? 12 : 5;
};
// TMEM columns: the S buffers at 0 and 128, O at 256 and (two groups) 384
constexpr uint32_t kTmemO = 256;

struct Maps {
    CUtensorMap k, v, kd, vd;
};

struct Bars {
    uint64_t full[12], empty[12];
    uint64_t s_full[2], p_full[2], p_halves[2], pv_done[2];  // p_halves: P by both groups
    uint64_t q_full, o_free, ml_full, drain;
};

// Shared memory: the swizzled operands first (1024-byte aligned), all of it
// dynamic, since the ring takes all that is left of the 227 KB.
template <int D>
struct Smem16 {
    unsigned char q[Shape<D>::kQBytes];
    unsigned char ring[Shape<D>::kSlots * Shape<D>::kTile];
    float2 ml[2][128];                      // (maximum, weight) of each group's rows
    Bars bars;
    AttnScan scan;
    uint32_t bad[4][ABG_MAX_SPAN / 32];     // drafts whose V holds an infinity or a NaN, of stretches in turn
    uint32_t tmem;
    int last[Shape<D>::kCopyWarps];         // last ring item that each copying warp has asked for (-1: none)
    volatile int gone;                      // a wait has given up
};
static_assert(sizeof(Smem16<64>) <= 227 * 1024 && sizeof(Smem16<128>) <= 227 * 1024 &&
                  sizeof(Smem16<256>) <= 227 * 1024,
              "shared memory of a block");

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
// Waits for the thread's loads.  x (a load's registers) may be read only after
// it, which the operands say; tmem_ld_also says it of further ones.
__device__ __forceinline__ void tmem_ld_wait(float (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
                   "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]),
                   "+f"(x[15]), "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]),
                   "+f"(x[22]), "+f"(x[23]), "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]),
                   "+f"(x[29]), "+f"(x[30]), "+f"(x[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_also(float (&x)[32]) {
    asm volatile(""
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
                   "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]),
                   "+f"(x[15]), "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]),
                   "+f"(x[22]), "+f"(x[23]), "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]),
                   "+f"(x[29]), "+f"(x[30]), "+f"(x[31]));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void cp16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
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
// the block has: the kernel then waits for its copies and products in flight,
// frees its TMEM and ends, with the device status word set.  Its units' entries
// are written all the same, since the joining launch goes by them.
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

// Which of a stretch's ring items holds V of its tile j (of n).  The order is the
// one the issuing warp first needs them.  Rows in both groups: K0 V0 K1 V1 ..;
// otherwise a step ahead: K0 K1 V0 K2 V1 .. V(n-1).
__device__ __forceinline__ int item_v(bool both, int j, int n) {
    return both || j == n - 1 ? 2 * j + 1 : 2 * j + 2;
}

// A ring slot and the phase of its item.
struct Place {
    int slot;
    uint32_t phase;
    __device__ __forceinline__ void skip(int items, int slots) {
        slot += items;
        if (items > slots) {
            phase ^= (slot / slots) & 1;
            slot %= slots;
        } else if (slot >= slots) {
            slot -= slots;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

template <typename T, int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) attn16_kernel(const __grid_constant__ AttnArgs p,
                                                                      const __grid_constant__ Maps maps, int box,
                                                                      int withhold) {
    using S = Shape<D>;
    constexpr int kKT = S::kKT, kSlots = S::kSlots, kCols = S::kCols, kRT = S::kRT, kGroups = S::kGroups;
    constexpr int kIssueWarp = 4 * kGroups, kCopyWarp = kIssueWarp + 1, kCopyWarps = S::kCopyWarps;
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem16<D> &sm = *reinterpret_cast<Smem16<D> *>(raw);
    Bars &bars = sm.bars;
    const abg_tree_attn_args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        sm.gone = 0;
        for (int i = 0; i < kSlots; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < 2; ++i)
            mbar_init(&bars.s_full[i], 1), mbar_init(&bars.p_full[i], 4), mbar_init(&bars.pv_done[i], 1),
                mbar_init(&bars.p_halves[i], 8);
        mbar_init(&bars.q_full, 4), mbar_init(&bars.o_free, 4 * kGroups);
        mbar_init(&bars.ml_full, 4 * kGroups), mbar_init(&bars.drain, 1);
        fence_mbar_init();
    }
    if (warp == kCopyWarp && lane < 4) {
        const CUtensorMap *map = lane == 0 ? &maps.k : lane == 1 ? &maps.v : lane == 2 ? &maps.kd : &maps.vd;
        asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    tc_before();
    grid_dep_wait();
    grid_dep_launch();
    AttnLine<kRT, kKT> line;
    line.template init<S::kThreads>(p, blockIdx.x, gridDim.x, sm.scan);
    __syncthreads();
    tc_after();
    const uint32_t tmem = sm.tmem;
    AttnSeg s{};
    bool live = true;

    if (warp >= kCopyWarp) {
        // ------------------------------------------------ the copying warps
        // Item i of the ring is brought by warp i % kCopyWarps: a tile of small
        // pages is many boxes, and a warp issues one at a time.
        // The lane's box of a tile: its row and page.  Taken before the wait
        // for the slot, so that the table's latency is not in the way.  The
        // first of these warps leaves the units' entries: it has the stretches
        // early, and registers to spare.
        bool left = false;
        struct At {
            int y, z;
        };
        const int page = static_cast<int>(a.page);
        auto where = [&](int t, int i) {
            At at{0, 0};
            if (t < s.ctiles) {
                const int key = t * kKT + i * box;
                if (key < s.req.len) {
                    const int j = key / page;
                    const int64_t id = a.table[static_cast<int64_t>(s.b) * a.width + j];
                    at.y = key - j * page;
                    at.z = id >= 0 && id < a.pages ? static_cast<int>(id * a.Hkv) + s.h : -1;  // -1: zeros
                }
            } else {
                at.y = s.req.n0 + (t - s.ctiles) * kKT + i * kDraftBox;
                at.z = s.h;
            }
            return at;
        };
        int first_item = 0, last = -1;  // last: this warp's last item so far
        auto bring = [&](int t, bool value, int item) {
            if (item == withhold) {  // the self-test: a copy that never comes
                live = false;
                return;
            }
            const bool cache = t < s.ctiles;
            const int step = cache ? box : kDraftBox, boxes = (tile_tokens<kKT>(s, t) + step - 1) / step;
            const CUtensorMap *map = cache ? (value ? &maps.v : &maps.k) : (value ? &maps.vd : &maps.kd);
            const int slot = item % kSlots;
            unsigned char *to = sm.ring + static_cast<uint32_t>(slot) * S::kTile;
            uint64_t *bar = &bars.full[slot];
            At at = where(t, lane);
            live = __all_sync(0xffffffffu, wait16(&bars.empty[slot], (item / kSlots + 1) & 1, &sm.gone));
            if (!live) return;
            if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * step) * D * 2);
            __syncwarp();
            for (int i = lane; i < boxes; i += 32) {
                if (i != lane) at = where(t, i);
#pragma unroll
                for (int cb = 0; cb < kCols; ++cb)
                    tma_3d(to + static_cast<uint32_t>(cb) * kKT * 128 + static_cast<uint32_t>(i * step) * 128, map,
                           64 * cb, at.y, at.z, bar);
            }
            last = item;
        };
        while (live && line.next(p, s)) {
            const bool both = s.rows > 128;
            const int n = s.t1 - s.t0;
            // the warp's items of the stretch, in order
            int i = (warp - kCopyWarp) - first_item % kCopyWarps;
            for (i += i < 0 ? kCopyWarps : 0; live && i < 2 * n; i += kCopyWarps) {
                const bool value = both ? i & 1 : i > 0 && (!(i & 1) || i == 2 * n - 1);
                const int j = both ? i >> 1 : !value ? (i + 1) >> 1 : i == 2 * n - 1 ? n - 1 : (i >> 1) - 1;
                bring(s.t0 + j, value, first_item + i);
            }
            first_item += 2 * n;
            if (warp == kCopyWarp && lane == 0) line.leave_entry(p, s, blockIdx.x, left);
        }
        if (lane == 0) sm.last[warp - kCopyWarp] = last;
        if (warp == kCopyWarp && lane == 0) {
            while (line.next(p, s)) line.leave_entry(p, s, blockIdx.x, left);  // after a wait that gave up
            line.end_entries(p, blockIdx.x, left);
        }
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------- the issuing warp
        // One elected lane does it all: every product waits on it, so that
        // it keeps its places in the ring instead of working them out.
        if (elect()) {
            constexpr uint32_t kQK = instr_desc<T>(128, kKT, false), kPV = instr_desc<T>(128, D, true);
            const uint64_t dq = smem_desc(smem_u32(sm.q), 16), dk = smem_desc(smem_u32(sm.ring), 16),
                           dv = smem_desc(smem_u32(sm.ring), kKT * 128);
            Place first{0, 0};          // of the stretch's first item
            uint32_t done = 3;          // bit b: next phase of buffer b's pv_done (the first wait passes)
            uint32_t weights = 0;       // of p_full; from bit 2 on of p_halves
            for (int seg = 0; live && line.next(p, s); ++seg) {
                const bool both = s.rows > 128;
                const int n = s.t1 - s.t0, steps = both ? 2 * n : n;
                Place k = first, v = first;
                v.skip(both || n == 1 ? 1 : 2, kSlots);
                // S of step i (buffer i & 1): row group i & 1 and tile i / 2, or tile i
                auto product = [&](int i) {
                    const int b = i & 1;
                    live = wait16(&bars.full[k.slot], k.phase, &sm.gone) &&
                           wait16(&bars.pv_done[b], done >> b & 1, &sm.gone);
                    if (!live) return;
                    done ^= 1u << b;
                    tc_after();
                    const uint64_t q = dq + (both && b ? S::kQTile >> 4 : 0u), kd = dk + k.slot * (S::kTile >> 4);
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
                        mma_ss(tmem + b * 128, q + (((d / 4) * (128 * 128) + (d % 4) * 32) >> 4),
                               kd + (((d / 4) * (kKT * 128) + (d % 4) * 32) >> 4), kQK, d > 0);
                    tc_commit(&bars.s_full[b]);
                    if (!both || b) {
                        tc_commit(&bars.empty[k.slot]);
                        k.skip(both || i > 0 ? 2 : 1, kSlots);
                    }
                };
                live = wait16(&bars.q_full, seg & 1, &sm.gone);
                if (live) product(0);
                if (live && steps > 1) product(1);
                const bool halves = kGroups == 2 && !both;
                bool upper = false;  // the second half's O has been written
                for (int i = 0; live && i < steps; ++i) {
                    const int b = i & 1, j = both ? i >> 1 : i, p_bit = halves ? b + 2 : b;
                    live = wait16(&bars.full[v.slot], v.phase, &sm.gone) &&
                           wait16(halves ? &bars.p_halves[b] : &bars.p_full[b], weights >> p_bit & 1, &sm.gone) &&
                           (i > 0 || seg == 0 || wait16(&bars.o_free, (seg - 1) & 1, &sm.gone));
                    if (!live) break;
                    weights ^= 1u << p_bit;
                    tc_after();
                    const uint64_t vd = dv + v.slot * (S::kTile >> 4);
                    const uint32_t o = tmem + kTmemO, w = tmem + b * 128;
                    // sums over `count` 16-token steps from step e0 on; past the
                    // tile's tokens there is no weight
                    const int count = (tile_tokens<kKT>(s, s.t0 + j) + 15) / 16;
                    auto sums = [&](uint32_t to, uint32_t from, int e0, int e1, bool add) {
#pragma unroll
                        for (int e = 0; e < kKT / 16; ++e)
                            if (e >= e0 && e < e1) mma_ts(to, from + (e - e0) * 8, vd + e * 128, kPV, add || e > e0);
                    };
                    if (halves) {
                        sums(o, w, 0, min(count, 4), i > 0);
                        if (count > 4) {
                            sums(o + 128, w + 64, 4, count, upper);
                            upper = true;
                        }
                    } else {
                        sums(o + (both && b ? 128u : 0u), w, 0, count, both ? i > 1 : i > 0);
                    }
                    tc_commit(&bars.pv_done[b]);
                    if (!both || b) {
                        tc_commit(&bars.empty[v.slot]);
                        v.skip(both || j + 2 != n ? 2 : 1, kSlots);
                    }
                    if (i + 2 < steps) product(i + 2);
                }
                first.skip(2 * n, kSlots);
            }
        }
    } else {
        // ------------------------------------------------- the softmax rows
        const int group = kGroups == 2 ? warp >> 2 : 0;
        // Weights are 2^(s - ref + kLift): of f16's 65504 the 2^8 that the
        // reference may be behind leaves 2^7, which keep a weight's 11 bits
        // down to 2^-21 of the largest instead of 2^-14, and half a unit of
        // those below at 2^-32 of it instead of 2^-25.  The weight sum and O
        // have the same factor, in every piece and group.  bf16 has f32's
        // exponents.
        constexpr float kLift = std::is_same_v<T, __half> ? 7.0f : 0.0f;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        int first_item = 0, seg = 0;
        // bit b: next phase of buffer b's s_full; phase of pv_done that the
        // buffer's last step completes
        uint32_t scores = 0, done = 3;
        // By one group: a stretch's Q, swizzled (16-byte chunk ch of row q at
        // chunk ch ^ (q % 8)), and its list of bad drafts, emptied.
        auto bring_q = [&](const AttnSeg &g, int of) {
            if ((tid & 127) < ABG_MAX_SPAN / 32) sm.bad[of & 3][tid & 127] = 0;
            for (int i = tid & 127; i < g.rows * (D / 8); i += 128) {
                const int q = i / (D / 8), ch = i % (D / 8), row = g.r0 + q;
                cp16(sm.q + (q / 128) * S::kQTile + (ch / 8) * (128 * 128) + (q % 128) * 128 + ((ch % 8) ^ (q % 8)) * 16,
                     static_cast<const T *>(a.q) +
                         ((static_cast<int64_t>(g.req.n0) + row / p.G) * a.Hq + g.h * p.G + row % p.G) * D + ch * 8);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.q_full);
        };
        AttnSeg next{};
        bool more = line.next(p, next);
        if (more && group == 0) bring_q(next, 0);
        for (; live && more; ++seg) {
            s = next;
            const bool both = s.rows > 128;
            const int n = s.t1 - s.t0, steps = both ? 2 * n : n;
            const int r = (tid & 127) + (both ? 128 * group : 0);  // row of the unit
            const bool busy = r - lane < s.rows, mine = r < s.rows;
            uint32_t *bad = sm.bad[seg & 3];
            const int64_t row = static_cast<int64_t>(s.req.n0) + (s.r0 + (mine ? r : 0)) / p.G;
            const uint64_t *seen = a.mask + row * a.words;
            float ref = -INFINITY, l = 0.0f;
            const uint32_t o_at = tmem + kTmemO + lanes;  // group 0's O
            const uint32_t o_mine = o_at + group * 128;
            // this group's steps, and its 64-token halves of their tiles
            const bool halves = kGroups == 2 && !both;
            const int h0 = halves ? group : 0, nh = halves ? 1 : kKT / 64;
            for (int i = both ? group : 0; i < steps; i += both ? 2 : 1) {
                const int b = i & 1, j = both ? i >> 1 : i, t = s.t0 + j;
                const bool drafts = t >= s.ctiles;
                const int tokens = tile_tokens<kKT>(s, t), key0 = (t - s.ctiles) * kKT;
                const uint32_t sbuf = tmem + b * 128 + lanes;
                live = __all_sync(0xffffffffu, wait16(&bars.s_full[b], scores >> b & 1, &sm.gone));
                if (!live) break;
                scores ^= 1u << b;
                tc_after();
                if (busy) {
                    // 64 scores at a time: the last ones are read for the maximum,
                    // then again for their weights, which keeps the row in 168
                    // registers
                    float x[64];
                    auto read = [&](int h) {
                        float(&lo)[32] = *reinterpret_cast<float(*)[32]>(x);
                        float(&hi)[32] = *reinterpret_cast<float(*)[32]>(x + 32);
                        tmem_ld32(sbuf + 64 * h, lo);
                        tmem_ld32(sbuf + 64 * h + 32, hi);
                        tmem_ld_wait(lo);
                        tmem_ld_also(hi);
                        if (drafts || tokens < kKT) {
                            uint64_t bits = ~0ull;
                            if (drafts) bits = key0 / 64 + h < a.words ? seen[key0 / 64 + h] : 0;
                            const int left = tokens - 64 * h;
                            if (left < 64) bits &= left > 0 ? (1ull << left) - 1 : 0;
#pragma unroll
                            for (int k = 0; k < 64; ++k)
                                if (!(bits >> k & 1)) x[k] = -INFINITY;
                        }
                    };
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int h = kKT / 64 - 1; h >= 0; --h) {
                        if (h >= nh) continue;
                        read(h0 + h);
#pragma unroll
                        for (int k = 0; k < 64; k += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e) top[e] = max3(top[e], x[k + e], x[k + 4 + e]);
                    }
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
                        if (i > (both ? 1 : 0)) {  // O holds this group's earlier steps
                            const int pb = both ? b : b ^ 1;  // the last one's buffer
                            live = __all_sync(0xffffffffu, wait16(&bars.pv_done[pb], done >> pb & 1, &sm.gone));
                            if (!live) break;
                            tc_after();
#pragma unroll 1
                            for (int k = 0; k < D; k += 32) {
                                float o[32];
                                tmem_ld32(o_mine + k, o);
                                tmem_ld_wait(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= f;
                                tmem_st32(o_mine + k, *reinterpret_cast<uint32_t(*)[32]>(o));
                            }
                        }
                    }
                    const float sub = ref == -INFINITY ? 0.0f : ref - kLift;
                    const float2 mul = make_float2(p.scale2, p.scale2), off = make_float2(-sub, -sub);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                    for (int h = 0; h < kKT / 64; ++h) {
                        if (h >= nh) continue;
                        if (h > 0) read(h0 + h);
                        uint32_t w[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float2 v = fma2(make_float2(x[2 * e], x[2 * e + 1]), mul, off);
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            sum[e & 1] = add2(sum[e & 1], v);
                            w[e] = pack2<T>(v.x, v.y);
                        }
                        tmem_st32(sbuf + 64 * h0 + 32 * h, w);
                    }
                    l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                    tmem_st_wait();
                }
                if ((drafts || tokens < kKT) && !(both && group)) {
                    // V rows past the tile's tokens hold what was there before,
                    // and a draft's V may hold an infinity or a NaN that only
                    // the rows that see it may get: 0 * NaN is NaN, so both are
                    // cleared here (the latter is added back at the end).  With
                    // rows in both groups the first clears for both: its
                    // product is issued first.
                    const int item = first_item + item_v(both, j, n), all = (tokens + 15) / 16 * 16;
                    live = __all_sync(0xffffffffu, wait16(&bars.full[item % kSlots], (item / kSlots) & 1, &sm.gone));
                    if (!live) break;
                    unsigned char *v = sm.ring + static_cast<uint32_t>(item % kSlots) * S::kTile;
                    for (int e = both ? tid & 127 : tid; e < all * (D / 8); e += both ? 128 : 128 * kGroups) {
                        const int q = e / (D / 8), ch = e % (D / 8);
                        uint4 *at = reinterpret_cast<uint4 *>(v + (ch / 8) * (kKT * 128) + q * 128 +
                                                              ((ch % 8) ^ (q % 8)) * 16);
                        if (q >= tokens) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else if (drafts) {
                            constexpr uint32_t kExp = std::is_same_v<T, __nv_bfloat16> ? 0x7f80u : 0x7c00u;
                            uint4 u = *at;
                            uint32_t *h = reinterpret_cast<uint32_t *>(&u);
                            bool hit = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((h[k] & kExp) == kExp) h[k] &= 0xffff0000u, hit = true;
                                if ((h[k] >> 16 & kExp) == kExp) h[k] &= 0xffffu, hit = true;
                            }
                            if (hit) {
                                *at = u;
                                atomicOr(&bad[(key0 + q) >> 5], 1u << ((key0 + q) & 31));
                            }
                        }
                    }
                    fence_async();
                }
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(halves ? &bars.p_halves[b] : &bars.p_full[b]);
                done ^= 1u << b;
            }
            if (!live) break;
            if (both && (n & 1)) scores ^= 2u >> group, done ^= 2u >> group;  // the other group's buffer
            first_item += 2 * n;
            // The group of the last step has seen its S, and with it the end of
            // every product that reads Q: the next stretch's Q comes before
            // this one's results are written.
            more = line.next(p, next);
            if (more && group == (both ? 1 : 0)) bring_q(next, seg + 1);
            // the products of the stretch's last steps
            live = wait16(&bars.pv_done[0], done & 1, &sm.gone) &&
                   (steps < 2 || wait16(&bars.pv_done[1], done >> 1 & 1, &sm.gone));
            live = __all_sync(0xffffffffu, live);
            if (!live) break;
            tc_after();
            float2 mine_ml = make_float2(ref, l), other_ml = make_float2(-INFINITY, 0.0f);
            if (kGroups == 2) {
                // (a product of this stretch is done, so every row has read
                // the last one's O, and sm.ml before it)
                if (halves) sm.ml[group][tid & 127] = mine_ml;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.ml_full);
                if (halves) {
                    live = __all_sync(0xffffffffu, wait16(&bars.ml_full, seg & 1, &sm.gone));
                    if (!live) break;
                    other_ml = sm.ml[group ^ 1][tid & 127];
                }
            }
            const bool whole = s.t0 == 0 && s.t1 == s.tiles;
            const int64_t piece = static_cast<int64_t>(2) * blockIdx.x + (s.t0 == 0);
            const int64_t at = (row * a.Hq + s.h * p.G + (s.r0 + (mine ? r : 0)) % p.G) * D;
            // after halves each group takes half of the columns of both O (of 64
            // columns the first takes all: a group sum has 64)
            const int k0 = halves && D > 64 ? group * (D / 2) : 0;
            const int k1 = !halves ? D : D > 64 ? k0 + D / 2 : group ? 0 : D;
            const float M = fmaxf(ref, other_ml.x);
            const float fm = l == 0.0f ? 0.0f : ex2(ref - M);
            const float fo = other_ml.y == 0.0f ? 0.0f : ex2(other_ml.x - M);
            const float L = l * fm + other_ml.y * fo;
            // in O's order: group 0's factor first
            const float f0 = halves && group ? fo : fm, f1 = halves && group ? fm : fo;
            if (busy) {
                float sums = 0.0f;
                const float scale = 1.0f / L;
#pragma unroll 1
                for (int k = k0; k < k1; k += 32) {
                    float o[32], o1[32];
                    __syncwarp();  // rows past the unit's have skipped ahead
                    tmem_ld32((halves ? o_at : o_mine) + k, o);
                    if (halves) tmem_ld32(o_at + 128 + k, o1);
                    tmem_ld_wait(o);
                    if (halves) tmem_ld_also(o1);
                    if (!mine) continue;
                    if (halves)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = (f0 == 0.0f ? 0.0f : o[e] * f0) + (f1 == 0.0f ? 0.0f : o1[e] * f1);
                    for (int w = 0; w < (s.req.T + 31) / 32; ++w)
                        for (uint32_t m = bad[w]; m; m &= m - 1) {
                            const int d = 32 * w + __ffs(static_cast<int>(m)) - 1;
                            if (!attn_sees(seen, d)) continue;
                            const T *vd = static_cast<const T *>(a.Vd) +
                                          (s.h * a.drafts + s.req.n0 + d) * static_cast<int64_t>(D) + k;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float v = static_cast<float>(vd[e]);
                                if (!(fabsf(v) < INFINITY)) o[e] += v;
                            }
                        }
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(p.part_o +
                                                        attn_piece_at<D, kRT, true>(piece, r, (k + e) / 4)) =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = L == 0.0f ? 0.0f : o[e] * scale;
                    if (a.gate)
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 g = *reinterpret_cast<const float4 *>(a.gate + at + k + e);
                            o[e] /= 1.0f + __expf(-g.x), o[e + 1] /= 1.0f + __expf(-g.y);
                            o[e + 2] /= 1.0f + __expf(-g.z), o[e + 3] /= 1.0f + __expf(-g.w);
                        }
                    if (a.y_type == ABG_SB_F32) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(static_cast<float *>(a.y) + at + k + e) =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + at + k + e) =
                                make_uint4(pack2<T>(o[e], o[e + 1]), pack2<T>(o[e + 2], o[e + 3]),
                                           pack2<T>(o[e + 4], o[e + 5]), pack2<T>(o[e + 6], o[e + 7]));
                    }
                    if (a.ysum) {
                        float sum = 0.0f;
#pragma unroll
                        for (int e = 0; e < 32; ++e) sum += o[e];
                        sums += sum;
                        if (k & 32) a.ysum[(at + k) / 64] = sums, sums = 0.0f;
                    }
                }
                if (mine && !whole && k0 == 0 && k1 > 0) p.part_ml[piece * kRT + r] = make_float2(M, L);
            }
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.o_free);
        }
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    tc_after();
    if (sm.gone) {
        // Whichever wait gave up, nothing that was asked for may arrive or read
        // after the block's end: the newest copy into each slot (the older ones
        // have been used), and the matrix instructions.
        if (warp == kCopyWarp && lane < kSlots) {
            int i = -1;
            for (int w = 0; w < kCopyWarps; ++w) i = max(i, sm.last[w]);
            while (i >= 0 && (i % kSlots != lane || i > sm.last[i % kCopyWarps])) --i;
            if (i >= 0) mbar_wait(&bars.full[lane], (i / kSlots) & 1);
        }
        if (warp == kIssueWarp && elect()) {  // the lane that issued them
            tc_commit(&bars.drain);
            mbar_wait(&bars.drain, 0);
        }
        __syncwarp();
    }
    if (warp == kIssueWarp)
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
cudaError_t go16(AttnArgs p, void *ws, bool early, bool pdl, int withhold, cudaStream_t stream) {
    using S = Shape<D>;
    static const cudaError_t attr =
        cudaFuncSetAttribute(attn16_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem16<D>));
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
    const AttnLayout l = attn_layout(C, S::kRT, D);
    unsigned char *w = static_cast<unsigned char *>(ws);
    p.part_o = reinterpret_cast<float *>(w + l.o);
    p.part_ml = reinterpret_cast<float2 *>(w + l.ml);
    p.split = reinterpret_cast<AttnSplit *>(w + l.split);
    attn_entries(p, C, S::kRT);
    const cudaError_t e =
        launch_kernel(attn16_kernel<T, D>, dim3(C), dim3(S::kThreads), sizeof(Smem16<D>), stream, early, p, m, box,
                      withhold);
    if (e != cudaSuccess) return e;
    return launch_join<T, D, S::kRT, true>(p, C, pdl, stream);
}

}  // namespace

size_t tree_attn16_bytes(int D) {
    const int rt = D == 64 ? Shape<64>::kRT : D == 128 ? Shape<128>::kRT : Shape<256>::kRT;
    return attn_layout(sm_count(), rt, D).total;
}

cudaError_t launch_tree_attn16(const AttnArgs &p, void *ws, bool early, bool pdl, int withhold, cudaStream_t stream) {
    auto of = [&](auto zero) {
        using T = decltype(zero);
        return p.a.D == 64    ? go16<T, 64>(p, ws, early, pdl, withhold, stream)
               : p.a.D == 128 ? go16<T, 128>(p, ws, early, pdl, withhold, stream)
                              : go16<T, 256>(p, ws, early, pdl, withhold, stream);
    };
    return p.a.type == ABG_SB_BF16 ? of(__nv_bfloat16{}) : of(__half{});
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
