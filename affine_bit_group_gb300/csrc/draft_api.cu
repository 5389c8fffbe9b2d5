// C ABI of the draft-verification calls (include/abg.h): argument validation
// and launches.  Everything that the host can see is refused here; lengths,
// tables and slots live on the GPU and are bounded by the kernels.
#include "draft.cuh"

#include <initializer_list>

using namespace abg;

namespace {

constexpr int64_t kMax32 = 0x7fffffff;

bool on(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

struct Span {
    uintptr_t lo, hi;
};
Span span(const void *p, int64_t count, size_t elem) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, p ? lo + static_cast<uintptr_t>(count) * elem : lo};
}
// No output may overlap an input or another output.
bool apart(std::initializer_list<Span> out, std::initializer_list<Span> in) {
    auto meet = [](Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; };
    for (auto o = out.begin(); o != out.end(); ++o) {
        for (auto p = out.begin(); p != o; ++p)
            if (meet(*o, *p)) return false;
        for (const Span &i : in)
            if (meet(*o, i)) return false;
    }
    return true;
}

bool known_type(int t) { return t >= ABG_SB_F32 && t <= ABG_SB_F16; }
int64_t elem(int t) { return t == ABG_SB_F32 ? 4 : 2; }
bool known_width(int64_t D) { return D == 64 || D == 128 || D == 256; }
// a product of positive factors that stays below 2^62
bool bounded(std::initializer_list<int64_t> f) {
    int64_t n = 1;
    for (int64_t v : f) {
        if (v < 0) return false;
        if (v > 0 && n > (int64_t(1) << 62) / v) return false;
        n *= v > 0 ? v : 1;
    }
    return true;
}
cudaStream_t to_stream(void *s) { return static_cast<cudaStream_t>(s); }

abg_status tree_attn(const abg_tree_attn_args *args, void *ws, int64_t ws_bytes, int withhold, void *stream) {
    if (!args) return ABG_EINVAL;
    const abg_tree_attn_args &a = *args;
    if (!known_type(a.type) || (a.y_type != a.type && a.y_type != ABG_SB_F32)) return ABG_EINVAL;
    if (a.ysum && a.y_type != ABG_SB_F32) return ABG_EINVAL;
    if (a.words < 1 || a.words > ABG_MAX_SPAN / 64 || a.B < 1 || a.B > kMax32 - 1 || a.N < 0 || a.N > kMax32 ||
        a.page < 1 || a.page > kMax32 || a.pages < 0 || a.pages > kMax32 || a.width < 0 || a.width > kMax32 ||
        !bounded({a.pages, a.Hkv}) || a.pages * a.Hkv > kMax32 || !bounded({a.B, a.width, 4}) || !bounded({a.width, a.page, 2}) || a.width * a.page > kMax32 || a.drafts < a.N || a.drafts > kMax32 ||
        a.max_span > 64 * a.words || !bounded({a.pages, a.page, a.Hkv, a.D, 4}) ||
        !bounded({a.drafts, a.Hq, a.D, 4}))
        return ABG_ESHAPE;
    int64_t need = 0;
    const abg_status st = abg_tree_attn_workspace(a.Hq, a.Hkv, a.D, a.max_span, a.type, &need);
    if (st != ABG_OK) return st;
    if (a.N == 0) return ABG_OK;
    if (!a.q || !a.lens || !a.cu || !a.Kd || !a.Vd || !a.mask || !a.y || !ws) return ABG_EINVAL;
    if ((a.width > 0 && !a.table) || (a.width > 0 && a.pages > 0 && (!a.Kc || !a.Vc))) return ABG_EINVAL;
    if (ws_bytes < need) return ABG_ESHAPE;
    for (const void *p : {a.q, a.Kc, a.Vc, a.Kd, a.Vd, static_cast<const void *>(a.gate),
                          static_cast<const void *>(a.y), static_cast<const void *>(ws)})
        if (!on(p, 16)) return ABG_EALIGN;
    if (!on(a.table, 4) || !on(a.lens, 4) || !on(a.cu, 4) || !on(a.mask, 8) || !on(a.ysum, 4)) return ABG_EALIGN;
    const int64_t te = elem(a.type), cache = a.pages * a.page * a.Hkv * a.D, io = a.N * a.Hq * a.D;
    if (!apart({span(a.y, io, elem(a.y_type)), span(a.ysum, io / 64, 4), span(ws, need, 1)},
               {span(a.q, io, te), span(a.Kc, cache, te), span(a.Vc, cache, te), span(a.table, a.B * a.width, 4),
                span(a.lens, a.B, 4), span(a.cu, a.B + 1, 4), span(a.Kd, a.Hkv * a.drafts * a.D, te),
                span(a.Vd, a.Hkv * a.drafts * a.D, te), span(a.mask, a.N * a.words, 8), span(a.gate, io, 4)}))
        return ABG_EALIAS;
    return cuda_status(launch_tree_attn(a, ws, early_launches(), withhold, to_stream(stream)), "tree_attn launch");
}

}  // namespace

extern "C" {

abg_status abg_page_plan(const int32_t *lens, const int32_t *add, const int32_t *cu, const int32_t *held,
                         const int64_t *ends, int32_t *ring, int32_t *table, int64_t *slots, int32_t *pos,
                         int32_t *lens_out, int32_t *held_out, int64_t *ends_out, int32_t *info, int64_t B, int64_t N,
                         int64_t page, int64_t width, int64_t ring_len, void *stream) {
    if (B < 1 || B > ABG_MAX_REQUESTS || N < 0 || N > kMax32 || page < 1 || page > kMax32 || width < 1 ||
        width > kMax32 || ring_len < 1 || ring_len > kMax32)
        return ABG_ESHAPE;
    if (!lens || !add || !cu || !held || !ends || !ring || !table || !lens_out || !held_out || !ends_out || !info ||
        (N > 0 && (!slots || !pos)))
        return ABG_EINVAL;
    for (const void *p : {static_cast<const void *>(lens), static_cast<const void *>(add),
                          static_cast<const void *>(cu), static_cast<const void *>(held),
                          static_cast<const void *>(ring), static_cast<const void *>(table),
                          static_cast<const void *>(pos), static_cast<const void *>(lens_out),
                          static_cast<const void *>(held_out), static_cast<const void *>(info)})
        if (!on(p, 4)) return ABG_EALIGN;
    if (!on(ends, 8) || !on(slots, 8) || !on(ends_out, 8)) return ABG_EALIGN;
    if (!apart({span(ring, ring_len, 4), span(table, B * width, 4), span(slots, N, 8), span(pos, N, 4),
                span(lens_out, B, 4), span(held_out, B, 4), span(ends_out, 2, 8), span(info, 2, 4)},
               {span(lens, B, 4), span(add, B, 4), span(cu, B + 1, 4), span(held, B, 4), span(ends, 2, 8)}))
        return ABG_EALIAS;
    const PagePlanArgs a{lens,     add,      cu,   held,                 ends,
                         ring,     table,    slots, pos,                 lens_out,
                         held_out, ends_out, info, static_cast<int>(B), static_cast<int>(N),
                         static_cast<int>(page), static_cast<int>(width), static_cast<int>(ring_len)};
    return cuda_status(launch_page_plan(a, early_launches(), to_stream(stream)), "page_plan launch");
}

abg_status abg_tree_plan(const int32_t *parent, const int32_t *lens, const int32_t *cu, uint64_t *mask, int32_t *pos,
                         int64_t B, int64_t N, int64_t words, void *stream) {
    if (B < 1 || B >= kMax32 || N < 0 || N > kMax32 || words < 1 || words > ABG_MAX_SPAN / 64) return ABG_ESHAPE;
    if (N == 0) return ABG_OK;
    if (!parent || !lens || !cu || !mask || !pos) return ABG_EINVAL;
    if (!on(parent, 4) || !on(lens, 4) || !on(cu, 4) || !on(pos, 4) || !on(mask, 8)) return ABG_EALIGN;
    if (!apart({span(mask, N * words, 8), span(pos, N, 4)},
               {span(parent, N, 4), span(lens, B, 4), span(cu, B + 1, 4)}))
        return ABG_EALIAS;
    return cuda_status(launch_tree_plan(parent, lens, cu, mask, pos, static_cast<int>(B), static_cast<int>(N),
                                        static_cast<int>(words), early_launches(), to_stream(stream)),
                       "tree_plan launch");
}

abg_status abg_kv_put(const abg_kv_put_args *args, void *stream) {
    if (!args) return ABG_EINVAL;
    abg_kv_put_args a = *args;
    if (!known_type(a.type) || (a.src_type != ABG_SB_F32 && a.src_type != a.type)) return ABG_EINVAL;
    if (a.N < 0 || a.N > kMax32 || a.src_rows < 0 || a.src_rows > kMax32 || a.Hkv < 1 || a.Hkv > 65536 ||
        !known_width(a.D) || a.page < 1 || a.page > kMax32 || a.pages < 0 || a.pages > kMax32 || a.q_row < 0 ||
        a.q_head < 0 || a.k_row < 0 || a.k_head < 0 || a.v_row < 0 || a.v_head < 0 ||
        !bounded({a.pages, a.page, a.Hkv, a.D, 4}) || !bounded({a.src_rows, a.k_row, 4}) ||
        !bounded({a.src_rows, a.v_row, 4}) || !bounded({a.Hkv, a.k_head, 4}) || !bounded({a.Hkv, a.v_head, 4}))
        return ABG_ESHAPE;
    if (a.q && (a.Hq < 1 || a.Hq > 65536 || !bounded({a.src_rows, a.q_row, 4}) || !bounded({a.Hq, a.q_head, 4})))
        return ABG_ESHAPE;
    if (!a.rows && a.src_rows < a.N) return ABG_ESHAPE;
    if ((a.cos != nullptr) != (a.sin != nullptr) || (a.q != nullptr) != (a.qo != nullptr)) return ABG_EINVAL;
    if (a.cos && (a.cos_rows < 1 || a.cos_rows > kMax32)) return ABG_ESHAPE;
    if (a.N == 0) return ABG_OK;
    if (!a.k || !a.v || !a.Kc || !a.Vc || (a.cos && !a.pos)) return ABG_EINVAL;
    const int64_t se = elem(a.src_type), te = elem(a.type);
    for (const void *p : {a.q, a.k, a.v, static_cast<const void *>(a.qo), static_cast<const void *>(a.Kc),
                          static_cast<const void *>(a.Vc), static_cast<const void *>(a.qn_w),
                          static_cast<const void *>(a.kn_w), static_cast<const void *>(a.cos),
                          static_cast<const void *>(a.sin)})
        if (!on(p, 16)) return ABG_EALIGN;
    for (int64_t st : {a.k_row, a.k_head, a.v_row, a.v_head, a.q ? a.q_row : 0, a.q ? a.q_head : 0})
        if (st * se % 16 != 0) return ABG_EALIGN;
    if (!on(a.rows, 4) || !on(a.slots, 8) || !on(a.pos, 4)) return ABG_EALIGN;
    auto source = [&](const void *p, int64_t row, int64_t head, int64_t H) {
        return span(p, a.src_rows > 0 ? (a.src_rows - 1) * row + (H - 1) * head + a.D : 0, se);
    };
    const int64_t cache = a.pages * a.page * a.Hkv * a.D;
    if (!apart({span(a.Kc, cache, te), span(a.Vc, cache, te), span(a.qo, a.q ? a.N * a.Hq * a.D : 0, te)},
               {source(a.k, a.k_row, a.k_head, a.Hkv), source(a.v, a.v_row, a.v_head, a.Hkv),
                source(a.q, a.q_row, a.q_head, a.q ? a.Hq : 1), span(a.rows, a.N, 4), span(a.slots, a.N, 8),
                span(a.pos, a.N, 4), span(a.qn_w, a.D, 4), span(a.kn_w, a.D, 4),
                span(a.cos, a.cos_rows * (a.D / 2), 4), span(a.sin, a.cos_rows * (a.D / 2), 4)}))
        return ABG_EALIAS;
    return cuda_status(launch_kv_put(a, early_launches(), to_stream(stream)), "kv_put launch");
}

abg_status abg_tree_attn_workspace(int64_t Hq, int64_t Hkv, int64_t D, int64_t max_span, int type, int64_t *bytes) {
    if (!bytes || !known_type(type)) return ABG_EINVAL;
    if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq > 65536 || !known_width(D) || max_span < 1 ||
        max_span > ABG_MAX_SPAN)
        return ABG_ESHAPE;
    *bytes = static_cast<int64_t>(tree_attn_bytes(static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(D),
                                                  static_cast<int>(max_span), type));
    return ABG_OK;
}

abg_status abg_tree_attn(const abg_tree_attn_args *args, void *ws, int64_t ws_bytes, void *stream) {
    return tree_attn(args, ws, ws_bytes, -1, stream);
}

abg_status abg_selftest_tree_attn_timeout(const abg_tree_attn_args *args, void *ws, int64_t ws_bytes, int item,
                                          void *stream) {
    if (item < 0 || (args && args->type == ABG_SB_F32)) return ABG_EINVAL;
    return tree_attn(args, ws, ws_bytes, item, stream);
}

abg_status abg_tree_accept_workspace(int64_t N, int64_t V, int64_t *bytes) {
    if (!bytes) return ABG_EINVAL;
    if (N < 0 || N > kMax32 || V < 1 || V > kMax32) return ABG_ESHAPE;
    *bytes = static_cast<int64_t>(tree_accept_bytes(N, V));
    return ABG_OK;
}

abg_status abg_tree_accept(const float *logits, int64_t ld, const int32_t *tok, const int32_t *parent,
                           const int32_t *cu, int32_t *best, int32_t *rows, int32_t *add, int32_t *last, int64_t B,
                           int64_t N, int64_t V, void *ws, int64_t ws_bytes, void *stream) {
    if (B < 1 || B >= kMax32 || ld < V || !bounded({N, ld, 4})) return ABG_ESHAPE;
    int64_t need = 0;
    const abg_status st = abg_tree_accept_workspace(N, V, &need);
    if (st != ABG_OK) return st;
    if (!cu || !add || !last || (N > 0 && (!logits || !tok || !parent || !best || !rows || !ws))) return ABG_EINVAL;
    if (ws_bytes < need) return ABG_ESHAPE;
    if (!on(logits, 4) || !on(tok, 4) || !on(parent, 4) || !on(cu, 4) || !on(best, 4) || !on(rows, 4) || !on(add, 4) ||
        !on(last, 4) || !on(ws, 8))
        return ABG_EALIGN;
    if (!apart({span(best, N, 4), span(rows, N, 4), span(add, B, 4), span(last, B, 4), span(ws, need, 1)},
               {span(logits, N > 0 ? (N - 1) * ld + V : 0, 4), span(tok, N, 4), span(parent, N, 4),
                span(cu, B + 1, 4)}))
        return ABG_EALIAS;
    return cuda_status(launch_tree_accept(logits, ld, tok, parent, cu, best, rows, add, last, static_cast<int>(B),
                                          static_cast<int>(N), V, ws, early_launches(), to_stream(stream)),
                       "tree_accept launch");
}

}  // extern "C"
