// C ABI of the quantised cache's calls (include/abg.h): argument validation and
// launches, as for the draft-verification calls.
#include "checks.cuh"
#include "draft.cuh"
#include "kvq.cuh"

using namespace abg;

namespace {

bool known_format(const abg_kvq_cache &c) {
    return (c.bits == 4 || c.bits == 8) && (c.group == 32 || c.group == 64);
}
bool cache_sizes(const abg_kvq_cache &c) {
    return c.page >= 1 && c.page <= kMax32 && c.pages >= 0 && c.pages <= kMax32 && c.Hkv >= 1 && c.Hkv <= 65536 &&
           known_width(c.D) && bounded({c.pages, c.page, c.Hkv, c.D, 4}) && bounded({c.pages, c.Hkv}) &&
           c.pages * c.Hkv <= kMax32 && c.pages * c.page * c.Hkv <= 2 * kMax32;
}
bool cache_aligned(const abg_kvq_cache &c) { return on(c.Kc, 16) && on(c.Ks, 16) && on(c.Vc, 16) && on(c.Vs, 16); }
struct CacheSpans {
    Span Kc, Ks, Vc, Vs;
};
CacheSpans spans_of(const abg_kvq_cache &c) {
    const int64_t rows = c.pages * c.page * c.Hkv, codes = rows * (c.D / 8), pairs = rows * (c.D / c.group);
    return {span(c.Kc, codes, static_cast<size_t>(c.bits)), span(c.Ks, pairs, 4),
            span(c.Vc, codes, static_cast<size_t>(c.bits)), span(c.Vs, pairs, 4)};
}

}  // namespace

extern "C" {

abg_status abg_kvq_put(const abg_kvq_put_args *args, void *stream) {
    if (!args) return ABG_EINVAL;
    const abg_kvq_put_args &a = *args;
    const abg_kvq_cache &c = a.c;
    if (!known_type(a.src_type) || !known_format(c)) return ABG_EINVAL;
    if (a.q && (!known_type(a.q_type) || (a.src_type != ABG_SB_F32 && a.q_type != a.src_type))) return ABG_EINVAL;
    if (!cache_sizes(c) || a.N < 0 || a.N > kMax32 || a.src_rows < 0 || a.src_rows > kMax32 || a.q_row < 0 ||
        a.q_head < 0 || a.k_row < 0 || a.k_head < 0 || a.v_row < 0 || a.v_head < 0 ||
        !bounded({a.src_rows, a.k_row, 4}) || !bounded({a.src_rows, a.v_row, 4}) || !bounded({c.Hkv, a.k_head, 4}) ||
        !bounded({c.Hkv, a.v_head, 4}))
        return ABG_ESHAPE;
    if (a.q && (a.Hq < 1 || a.Hq > 65536 || !bounded({a.src_rows, a.q_row, 4}) || !bounded({a.Hq, a.q_head, 4}) ||
                !bounded({a.N, a.Hq, c.D, 4})))
        return ABG_ESHAPE;
    if (!a.rows && a.src_rows < a.N) return ABG_ESHAPE;
    if ((a.cos != nullptr) != (a.sin != nullptr) || (a.q != nullptr) != (a.qo != nullptr)) return ABG_EINVAL;
    if (a.cos && (a.cos_rows < 1 || a.cos_rows > kMax32)) return ABG_ESHAPE;
    if (a.N == 0) return ABG_OK;
    if (!a.k || !a.v || (a.cos && !a.pos) || (c.pages > 0 && (!c.Kc || !c.Ks || !c.Vc || !c.Vs))) return ABG_EINVAL;
    const int64_t se = elem(a.src_type);
    for (const void *p : {a.q, a.k, a.v, static_cast<const void *>(a.qo), static_cast<const void *>(a.qn_w),
                          static_cast<const void *>(a.kn_w), static_cast<const void *>(a.cos),
                          static_cast<const void *>(a.sin)})
        if (!on(p, 16)) return ABG_EALIGN;
    for (int64_t st : {a.k_row, a.k_head, a.v_row, a.v_head, a.q ? a.q_row : 0, a.q ? a.q_head : 0})
        if (st * se % 16 != 0) return ABG_EALIGN;
    if (!cache_aligned(c) || !on(a.rows, 4) || !on(a.slots, 8) || !on(a.pos, 4)) return ABG_EALIGN;
    auto source = [&](const void *p, int64_t row, int64_t head, int64_t H) {
        return span(p, a.src_rows > 0 ? (a.src_rows - 1) * row + (H - 1) * head + c.D : 0, se);
    };
    const CacheSpans s = spans_of(c);
    const int64_t half = c.D / 2;
    if (!apart({s.Kc, s.Ks, s.Vc, s.Vs, span(a.qo, a.q ? a.N * a.Hq * c.D : 0, elem(a.q ? a.q_type : 0))},
               {source(a.k, a.k_row, a.k_head, c.Hkv), source(a.v, a.v_row, a.v_head, c.Hkv),
                source(a.q, a.q_row, a.q_head, a.q ? a.Hq : 1), span(a.rows, a.N, 4), span(a.slots, a.N, 8),
                span(a.pos, a.N, 4), span(a.qn_w, c.D, 4), span(a.kn_w, c.D, 4),
                span(a.cos, a.cos ? a.cos_rows * half : 0, 4), span(a.sin, a.cos ? a.cos_rows * half : 0, 4)}))
        return ABG_EALIAS;
    return cuda_status(launch_kvq_put(a, early_launches(), to_stream(stream)), "kvq_put launch");
}

abg_status abg_kvq_get(const abg_kvq_get_args *args, void *stream) {
    if (!args) return ABG_EINVAL;
    const abg_kvq_get_args &a = *args;
    const abg_kvq_cache &c = a.c;
    if (!known_type(a.type) || !known_format(c)) return ABG_EINVAL;
    if (!cache_sizes(c) || a.N < 0 || a.N > kMax32 || a.k_row < 0 || a.k_head < 0 || a.v_row < 0 || a.v_head < 0 ||
        !bounded({a.N, a.k_row, 4}) || !bounded({a.N, a.v_row, 4}) || !bounded({c.Hkv, a.k_head, 4}) ||
        !bounded({c.Hkv, a.v_head, 4}) || !bounded({a.N, c.Hkv, c.D}))
        return ABG_ESHAPE;
    if (a.N == 0) return ABG_OK;
    if ((!a.k && !a.v) || (c.pages > 0 && ((a.k && (!c.Kc || !c.Ks)) || (a.v && (!c.Vc || !c.Vs))))) return ABG_EINVAL;
    const int64_t e = elem(a.type);
    if (!on(a.k, 16) || !on(a.v, 16) || !on(a.slots, 8) || !cache_aligned(c)) return ABG_EALIGN;
    for (int64_t st : {a.k ? a.k_row : 0, a.k ? a.k_head : 0, a.v ? a.v_row : 0, a.v ? a.v_head : 0})
        if (st * e % 16 != 0) return ABG_EALIGN;
    if ((a.k && !rows_apart({a.k_row, a.k_head}, a.N, c.Hkv, c.D)) ||
        (a.v && !rows_apart({a.v_row, a.v_head}, a.N, c.Hkv, c.D)))
        return ABG_EALIAS;
    const int64_t ke = (c.Hkv - 1) * a.k_head + c.D, ve = (c.Hkv - 1) * a.v_head + c.D;  // of one row's heads
    const Span ks = span(a.k, (a.N - 1) * a.k_row + ke, static_cast<size_t>(e)),
               vs = span(a.v, (a.N - 1) * a.v_row + ve, static_cast<size_t>(e)), none{0, 0};
    const CacheSpans s = spans_of(c);
    for (const Span &out : {a.k ? ks : none, a.v ? vs : none})
        if (!apart({out}, {s.Kc, s.Ks, s.Vc, s.Vs, span(a.slots, a.N, 8)})) return ABG_EALIAS;
    if (a.k && a.v && !apart({ks, vs}, {})) {
        // k and v of one buffer
        const bool k_first = ks.lo < vs.lo;
        const int64_t off = static_cast<int64_t>(k_first ? vs.lo - ks.lo : ks.lo - vs.lo) / e;
        const RowStrides k{a.k_row, a.k_head}, v{a.v_row, a.v_head};
        if (!(k_first ? rows_between(off, k, v, a.N, c.Hkv, c.D) : rows_between(off, v, k, a.N, c.Hkv, c.D)))
            return ABG_EALIAS;
    }
    return cuda_status(launch_kvq_get(a, early_launches(), to_stream(stream)), "kvq_get launch");
}

abg_status abg_kvq_attn_workspace(const abg_kvq_cache *c, int64_t Hq, int64_t max_span, int type, int64_t *bytes) {
    if (!bytes || !c || !known_type(type) || !known_format(*c)) return ABG_EINVAL;
    if (c->Hkv < 1 || Hq < c->Hkv || Hq % c->Hkv != 0 || Hq > 65536 || !known_width(c->D) || max_span < 1 ||
        max_span > ABG_MAX_SPAN)
        return ABG_ESHAPE;
    *bytes = static_cast<int64_t>(kvq_attn_bytes(*c, Hq, max_span, type));
    return ABG_OK;
}

abg_status abg_kvq_attn(const abg_kvq_attn_args *args, void *ws, int64_t ws_bytes, void *stream) {
    if (!args) return ABG_EINVAL;
    const abg_kvq_attn_args &a = *args;
    const abg_kvq_cache &c = a.c;
    if (!known_type(a.type) || !known_format(c) || (a.y_type != a.type && a.y_type != ABG_SB_F32)) return ABG_EINVAL;
    if (a.ysum && a.y_type != ABG_SB_F32) return ABG_EINVAL;
    if (!cache_sizes(c) || a.words < 1 || a.words > ABG_MAX_SPAN / 64 || a.B < 1 || a.B > kMax32 - 1 || a.N < 0 ||
        a.N > kMax32 || a.width < 0 || a.width > kMax32 || !bounded({a.B, a.width, 4}) ||
        // (a kernel's token numbers pass the last cached one by up to 1535)
        !bounded({a.width, c.page, 2}) || a.width * c.page > kMax32 - 2047 || a.drafts < a.N || a.drafts > kMax32 ||
        a.max_span > 64 * a.words || a.Hq < 1 || a.Hq > 65536 || !bounded({a.drafts, a.Hq, c.D, 4}))
        return ABG_ESHAPE;
    int64_t need = 0;
    const abg_status st = abg_kvq_attn_workspace(&c, a.Hq, a.max_span, a.type, &need);
    if (st != ABG_OK) return st;
    if (a.N == 0) return ABG_OK;
    if (!a.q || !a.lens || !a.cu || !a.Kd || !a.Vd || !a.mask || !a.y || !ws) return ABG_EINVAL;
    if ((a.width > 0 && !a.table) || (a.width > 0 && c.pages > 0 && (!c.Kc || !c.Ks || !c.Vc || !c.Vs))) return ABG_EINVAL;
    if (ws_bytes < need) return ABG_ESHAPE;
    for (const void *p : {a.q, a.Kd, a.Vd, static_cast<const void *>(a.gate), static_cast<const void *>(a.y),
                          static_cast<const void *>(ws)})
        if (!on(p, 16)) return ABG_EALIGN;
    if (!cache_aligned(c) || !on(a.table, 4) || !on(a.lens, 4) || !on(a.cu, 4) || !on(a.mask, 8) || !on(a.ysum, 4))
        return ABG_EALIGN;
    const int64_t te = elem(a.type), io = a.N * a.Hq * c.D;
    const CacheSpans s = spans_of(c);
    if (!apart({span(a.y, io, elem(a.y_type)), span(a.ysum, io / 64, 4), span(ws, need, 1)},
               {span(a.q, io, te), s.Kc, s.Ks, s.Vc, s.Vs, span(a.table, a.B * a.width, 4), span(a.lens, a.B, 4),
                span(a.cu, a.B + 1, 4), span(a.Kd, c.Hkv * a.drafts * c.D, te),
                span(a.Vd, c.Hkv * a.drafts * c.D, te), span(a.mask, a.N * a.words, 8), span(a.gate, io, 4)}))
        return ABG_EALIAS;
    return cuda_status(launch_kvq_attn(a, ws, early_launches(), to_stream(stream)), "kvq_attn launch");
}

}  // extern "C"
