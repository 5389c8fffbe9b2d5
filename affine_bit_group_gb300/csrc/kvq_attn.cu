// kvq_attn: which of its kernels a call takes (kvq_attn.cuh).
#include "abg_kernels.cuh"
#include "kvq_attn.cuh"

#include <cmath>

namespace abg {

template <>
cudaError_t kvq_attn_launch<64, 4>(const KvqAttnArgs &, int, int, bool, void *, bool, bool, cudaStream_t);
template <>
cudaError_t kvq_attn_launch<64, 8>(const KvqAttnArgs &, int, int, bool, void *, bool, bool, cudaStream_t);
template <>
cudaError_t kvq_attn_launch<128, 4>(const KvqAttnArgs &, int, int, bool, void *, bool, bool, cudaStream_t);
template <>
cudaError_t kvq_attn_launch<128, 8>(const KvqAttnArgs &, int, int, bool, void *, bool, bool, cudaStream_t);
template <>
cudaError_t kvq_attn_launch<256, 4>(const KvqAttnArgs &, int, int, bool, void *, bool, bool, cudaStream_t);
template <>
cudaError_t kvq_attn_launch<256, 8>(const KvqAttnArgs &, int, int, bool, void *, bool, bool, cudaStream_t);

size_t kvq_attn_bytes(const abg_kvq_cache &c, int64_t Hq, int64_t max_span, int type) {
    const int rt = kvq_row_tile(c.D, Hq / c.Hkv * max_span);
    const bool split = type != ABG_SB_BF16;
    auto bytes = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return c.bits == 4 ? kvq_by_rows<D, 4>(c.group, rt, split, KvqBytes{})
                           : kvq_by_rows<D, 8>(c.group, rt, split, KvqBytes{});
    };
    return c.D == 64    ? bytes(std::integral_constant<int, 64>{})
           : c.D == 128 ? bytes(std::integral_constant<int, 128>{})
                        : bytes(std::integral_constant<int, 256>{});
}

cudaError_t launch_kvq_attn(const abg_kvq_attn_args &a, void *ws, bool pdl, cudaStream_t stream) {
    KvqAttnArgs x{};
    abg_tree_attn_args &t = x.p.a;
    t.q = a.q, t.table = a.table, t.lens = a.lens, t.cu = a.cu, t.Kd = a.Kd, t.Vd = a.Vd, t.mask = a.mask;
    t.gate = a.gate, t.y = a.y, t.ysum = a.ysum;
    t.B = a.B, t.N = a.N, t.Hq = a.Hq, t.Hkv = a.c.Hkv, t.D = a.c.D, t.page = a.c.page, t.pages = a.c.pages;
    t.width = a.width, t.drafts = a.drafts, t.words = a.words, t.max_span = a.max_span;
    t.type = a.type, t.y_type = a.y_type;
    x.p.G = static_cast<int>(a.Hq / a.c.Hkv);
    x.p.scale2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.c.D)));
    x.Kc = static_cast<const unsigned char *>(a.c.Kc), x.Vc = static_cast<const unsigned char *>(a.c.Vc);
    x.Ks = static_cast<const unsigned char *>(a.c.Ks), x.Vs = static_cast<const unsigned char *>(a.c.Vs);
    // (without pages nothing is read, but a copy of no bytes still has an address)
    if (a.c.pages == 0) x.Kc = x.Vc = x.Ks = x.Vs = static_cast<const unsigned char *>(a.q);
    kvq_page_division(x, static_cast<uint32_t>(a.c.page));
    const bool early = pdl && !capturing(stream), split = a.type != ABG_SB_BF16;
    const int rt = kvq_row_tile(a.c.D, x.p.G * a.max_span), group = a.c.group;
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return a.c.bits == 4 ? kvq_attn_launch<D, 4>(x, group, rt, split, ws, early, pdl, stream)
                             : kvq_attn_launch<D, 8>(x, group, rt, split, ws, early, pdl, stream);
    };
    return a.c.D == 64    ? go(std::integral_constant<int, 64>{})
           : a.c.D == 128 ? go(std::integral_constant<int, 128>{})
                          : go(std::integral_constant<int, 256>{});
}

}  // namespace abg
