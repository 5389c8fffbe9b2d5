"""The quantised cache's calls on the GPU against their plain forms: codes,
factors and values read back equal, the attention within bounds derived from its
roundings."""
from __future__ import annotations

import numpy as np
import pytest

import draft_ref
import kvq_ref as ref
from helpers import dev, host
from test_gpu_9_draft import TYPES, U32, UNIT, bits_of, i32, i64, parents, wide

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
abg = pytest.importorskip("affine_bit_group_gb300")


def as_cache(Kw, Kp, Vw, Vp):
    return abg.KvqCache(*(dev(a.view(np.int32)) if a.dtype == np.uint32 else dev(a) for a in (Kw, Kp, Vw, Vp)))


def arrays(cache):
    return [host(cache[0]).view(np.uint32), host(cache[1]), host(cache[2]).view(np.uint32), host(cache[3])]


def same_bits(got, want, what=""):
    view = {4: np.uint32, 2: np.uint16}[want.dtype.itemsize]
    g, w = np.ascontiguousarray(got).view(view), np.ascontiguousarray(want).view(view)
    bad = np.argwhere(g != w)
    assert not len(bad), (what, len(bad), g.size, bad[:5], g[tuple(bad[0])], w[tuple(bad[0])])


# ---------------------------------------------------------------- kvq_put ----
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("kind,qkind,N,Hq,Hkv,D,page,norm,rope", [
    ("f32", "f32", 1, 4, 4, 64, 1, True, True), ("f32", "bf16", 37, 6, 3, 64, 7, True, True),
    ("f32", "f16", 130, 16, 4, 128, 16, True, False), ("f32", "f32", 5, 8, 2, 256, 100, False, True),
    ("bf16", "bf16", 64, 3, 1, 128, 48, True, True), ("f16", "f16", 33, 5, 5, 256, 16, True, True),
    ("f32", "bf16", 300, 8, 1, 256, 16, True, True), ("bf16", "bf16", 41, 2, 2, 64, 5, False, False)])
def test_kvq_put_is_its_steps_one_by_one(bits, group, kind, qkind, N, Hq, Hkv, D, page, norm, rope):
    rng = np.random.default_rng([N, Hq, D, page, bits, group])
    pages = -(-N // page) + 1
    qkv = torch.from_numpy((1.5 * rng.standard_normal((N, Hq + 2 * Hkv, D))).astype(np.float32)).to(TYPES[kind])
    slots = rng.permutation(pages * page)[:N].astype(np.int64)
    drop = rng.random(N) < 0.2
    slots[drop] = rng.choice([-1, -2**40, pages * page, 2**40], drop.sum())
    shape = (pages, Hkv, page)
    old = [rng.integers(0, 2**32, (*shape, D * bits // 32), dtype=np.uint32),
           rng.standard_normal((*shape, D // group, 2)).astype(np.float16)] * 2
    cache = as_cache(*old)
    qo = torch.full((N, Hq, D), 7.0, dtype=TYPES[qkind], device="cuda")
    w = [(1 + 0.1 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2)]
    ang = rng.uniform(0, 6.28, (2 * N, D // 2))
    cs = [np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)] if rope else [None, None]
    pos = rng.integers(0, 2 * N, N)
    d = qkv.cuda()
    opt = lambda x: None if x is None else dev(x)  # noqa: E731
    for _ in range(2):  # it can be repeated
        abg.kvq_put(d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], cache, slots=i64(slots), q=d[:, :Hq], qo=qo, qn_w=opt(w[0]),
                    kn_w=opt(w[1]), cos=opt(cs[0]), sin=opt(cs[1]), pos=i32(pos) if rope else None)
    x = qkv.float().numpy()
    q, k = ref.rows(x[:, :Hq], w[0], *cs, pos, 1e-6), ref.rows(x[:, Hq:Hq + Hkv], w[1], *cs, pos, 1e-6)
    want = [a.copy() for a in old]
    kept = (slots >= 0) & (slots < pages * page)
    at = slots[kept]
    for i, rows in ((0, k), (2, x[:, Hq + Hkv:])):
        words, pairs = ref.quantise(rows, bits, group)
        want[i][at // page, :, at % page] = words[kept]
        want[i + 1][at // page, :, at % page] = pairs[kept]
    for got, exp, what in zip(arrays(cache), want, ("Kc", "Ks", "Vc", "Vs")):
        same_bits(got, exp, what)
    assert torch.equal(qo.cpu(), torch.from_numpy(q).to(TYPES[qkind]))
    # what is held is within half a scale, the bias's rounding and 2^-11 of the range
    words, pairs = ref.quantise(k, bits, group)
    got, _ = ref.values(words, pairs, bits)
    g = k.astype(np.float64).reshape(N, Hkv, -1, group)
    room = 0.5 * pairs[..., :1].astype(np.float64) + (np.abs(g).max(-1, keepdims=True) + np.ptp(g, -1)[..., None]) * 2.0**-11
    assert np.all(np.abs(got.reshape(g.shape) - g) <= room * (1 + 1e-6) + 2.0**-24)  # (2^-25: f16's smallest, of both)


@pytest.mark.parametrize("kind,qkind,N,Hq,Hkv,D,page,bits,group", [
    ("f32", "bf16", 9001, 3, 1, 128, 16, 4, 64), ("bf16", "bf16", 3001, 5, 5, 64, 7, 8, 32),
    ("f32", "f32", 1100, 16, 4, 256, 48, 4, 32), ("f16", "f16", 1301, 7, 2, 256, 1, 8, 64),
    ("f32", "f16", 17, 512, 512, 64, 5, 4, 64)])
def test_kvq_put_of_more_units_than_warps(kind, qkind, N, Hq, Hkv, D, page, bits, group):
    test_kvq_put_is_its_steps_one_by_one(bits, group, kind, qkind, N, Hq, Hkv, D, page, True, True)


@pytest.mark.parametrize("kind,qkind", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 9, 3), (128, 4, 2), (256, 2, 1)])
def test_kvq_put_in_one_call_and_in_small_ones(kind, qkind, D, Hq, Hkv):
    """Rows and positions that there are not among them."""
    rng = np.random.default_rng([D, Hq])
    N, R, P, pages, page = 6007, 501, 90, 400, 16
    qkv = torch.from_numpy(rng.standard_normal((R, Hq + 2 * Hkv, D)).astype(np.float32)).to(TYPES[kind]).cuda()
    rows, pos = rng.integers(0, R, N), rng.integers(0, P, N)
    rows[rng.random(N) < 0.2] = -1
    rows[::97], rows[::89] = R, -2**31
    pos[::31], pos[::37] = P, -1
    slots = rng.permutation(pages * page)[:N]
    slots[::41] = -5
    rows, pos, slots = i32(rows), i32(pos), i64(slots)
    w, cos, sin = (dev(rng.standard_normal(n).astype(np.float32)) for n in (D, P * D // 2, P * D // 2))
    got = []
    for step in (N, 50):
        cache = abg.kvq_cache(pages, Hkv, page, D, 8, 32)
        qo = torch.full((N, Hq, D), 7.0, dtype=TYPES[qkind], device="cuda")
        for n in range(0, N, step):
            s = slice(n, n + step)
            abg.kvq_put(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cache, slots=slots[s], rows=rows[s].clone(), q=qkv[:, :Hq],
                        qo=qo[s], qn_w=w, kn_w=w, cos=cos, sin=sin, pos=pos[s].clone())
        got.append([*cache, qo])
    for one, many in zip(*got):
        same_bits(host(one.view(torch.int16)), host(many.view(torch.int16)), "one call")
    assert bool((got[0][4][host(rows) == -1] == 7.0).all()) and bool(got[0][4][host(rows) >= 0].float().abs().sum() != 0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_kvq_put_of_odd_groups(bits, group, D):
    """Equal values, zeros, tiny and huge ranges, an offset far above the range,
    NaN, infinities and magnitudes past f16: the rule's factors, group by group."""
    rng = np.random.default_rng([bits, group, D])
    rows = []
    for fill in (0.0, -0.0, 3.25, -1e-7, 65504.0, 65519.0, -65505.0, 1e30, np.nan, np.inf, -np.inf):
        x = rng.standard_normal(D)
        x[rng.integers(0, D)] = fill  # one value of one group
        rows += [np.full(D, fill), x]
    rows += [rng.standard_normal(D) * s for s in (1e-30, 1e-9, 1e-7, 1e-5, 1e4, 2e4)]
    rows += [100 + rng.standard_normal(D) * s for s in (1e-3, 0.02, 0.3)]
    rows += [np.where(np.arange(D) % 2, 65504.0, -65504.0), np.where(np.arange(D) % group, 6e-8, 0.0)]
    x = np.array(rows).astype(np.float32)[:, None]
    cache = abg.kvq_cache(1, 1, len(x), D, bits, group)
    abg.kvq_put(dev(x), dev(x[::-1]), cache)
    for got, exp, what in zip(arrays(cache), [*ref.quantise(x, bits, group), *ref.quantise(x[::-1], bits, group)],
                              ("Kc", "Ks", "Vc", "Vs")):
        same_bits(got[0, 0], exp[:, 0], what)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_kvq_put_takes_draft_rows_by_index(kind, bits, group):
    rng = np.random.default_rng(3)
    T, Hkv, D, R = TYPES[kind], 3, 128, 29
    Kd, Vd = (torch.from_numpy(rng.standard_normal((Hkv, R, D))).to(T).cuda() for _ in range(2))
    cache = abg.kvq_cache(4, Hkv, 10, D, bits, group)
    rows = np.array([0, 28, 5, -1, 29, 6, 2**31 - 1, 7], np.int32)
    slots = np.array([39, 0, 11, 12, 13, -1, 14, 25], np.int64)
    abg.kvq_put(Kd.transpose(0, 1), Vd.transpose(0, 1), cache, rows=i32(rows), slots=i64(slots))
    for i, src in ((0, Kd), (2, Vd)):
        words, pairs = ref.quantise(src.float().cpu().numpy(), bits, group)
        want = [np.zeros((4, Hkv, 10, D * bits // 32), np.uint32), np.zeros((4, Hkv, 10, D // group, 2), np.float16)]
        for r, s in zip(rows, slots):
            if 0 <= r < R and 0 <= s < 40:
                want[0][s // 10, :, s % 10], want[1][s // 10, :, s % 10] = words[:, r], pairs[:, r]
        same_bits(arrays(cache)[i], want[0])
        same_bits(arrays(cache)[i + 1], want[1])


def test_kvq_put_position_outside_the_rotation_table_is_held_as_nan():
    k = torch.ones((3, 1, 64), device="cuda")
    cache = abg.kvq_cache(1, 1, 3, 64)
    cs = torch.ones((5, 32), device="cuda")
    abg.kvq_put(k, k, cache, cos=cs, sin=torch.zeros_like(cs), pos=i32([4, 5, -1]))
    ko, vo = torch.zeros_like(k), torch.zeros_like(k)
    abg.kvq_get(cache, ko, vo)
    assert torch.equal(ko[0], k[0]) and torch.isnan(ko[1:]).all() and torch.equal(vo, k)


# ---------------------------------------------------------------- kvq_get ----
def random_cache(rng, pages, Hkv, page, D, bits, group):
    def part():
        x = rng.standard_normal((pages, Hkv, page, D)) * np.linspace(0.5, 2, D) + rng.standard_normal((1, Hkv, 1, D))
        return ref.quantise(x.astype(np.float32), bits, group)

    return [*part(), *part()]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group,D,Hkv,page,N", [
    (4, 64, 64, 1, 1, 1), (4, 32, 64, 3, 7, 50), (8, 64, 128, 4, 16, 333), (4, 64, 128, 2, 16, 1000), (8, 32, 256, 2, 100, 77),
    (4, 32, 256, 5, 48, 129), (8, 64, 64, 2, 33, 70)])
def test_kvq_get(kind, bits, group, D, Hkv, page, N):
    rng = np.random.default_rng([bits, group, D, N])
    pages = 9
    parts = random_cache(rng, pages, Hkv, page, D, bits, group)
    cache = as_cache(*parts)
    slots = rng.integers(0, pages * page, N)  # some slots several times
    slots[rng.random(N) < 0.1] = rng.choice([-1, pages * page, 2**40])
    ok = (slots >= 0) & (slots < pages * page)
    at = np.where(ok, slots, 0)
    T = TYPES[kind]
    want = []
    for w, p in (parts[:2], parts[2:]):
        v, _ = ref.values(w, p, bits)
        v = np.where(ok[:, None, None], v[at // page, :, at % page], 0.0).astype(np.float32)  # rounded once
        want.append(torch.from_numpy(v).to(T))
    k, v = (torch.full((N + 2, Hkv, D), 7.0, dtype=T, device="cuda") for _ in range(2))
    abg.kvq_get(cache, k, v, slots=i64(slots))
    for got, exp in ((k, want[0]), (v, want[1])):
        assert torch.equal(got[:N].cpu(), exp) and (got[N:] == 7).all()
    # rows inside other rows of one buffer, heads first, one of the two alone
    both = torch.full((N, 2 * Hkv + 1, D), 7.0, dtype=T, device="cuda")
    abg.kvq_get(cache, both[:, Hkv + 1:], both[:, :Hkv], slots=i64(slots))
    assert torch.equal(both[:, Hkv + 1:].cpu(), want[0]) and torch.equal(both[:, :Hkv].cpu(), want[1])
    assert (both[:, Hkv] == 7).all()
    heads = torch.full((Hkv, N + 1, D), 7.0, dtype=T, device="cuda")
    abg.kvq_get(cache, None, heads.transpose(0, 1), slots=i64(slots))
    assert torch.equal(heads[:, :N].transpose(0, 1).cpu(), want[1]) and (heads[:, N] == 7).all()
    abg.kvq_get(cache, k[:, :, :], None, slots=i64(slots[::-1].copy()))
    assert torch.equal(k[:N].cpu(), want[0].flip(0))


def test_kvq_get_without_slots_and_of_every_code():
    """Every 8-bit code and every nibble at every place of a word; rows in order."""
    for bits in (4, 8):
        rng = np.random.default_rng(bits)
        page, D = 64, 128
        words = rng.integers(0, 2**32, (3, 2, page, D * bits // 32), dtype=np.uint32)
        pairs = rng.standard_normal((3, 2, page, 2, 2)).astype(np.float16)  # negative scales too
        cache = as_cache(words, pairs, words[::-1].copy(), pairs[::-1].copy())
        k, v = (torch.empty((3 * page, 2, D), device="cuda") for _ in range(2))
        abg.kvq_get(cache, k, v)
        for got, w, p in ((k, words, pairs), (v, words[::-1], pairs[::-1])):
            want = ref.values(w, p, bits)[0].astype(np.float32).transpose(0, 2, 1, 3).reshape(3 * page, 2, D)
            assert np.array_equal(host(got), want)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("Hkv", [1, 2, 3])
@pytest.mark.parametrize("N", [1, 2, 5])
def test_kvq_get_into_one_buffer(kind, Hkv, N):
    """k and v between one another in one buffer: heads in turn (in rows with room at
    their end too), heads before rows with k and v in turn or side by side, and every
    other place as it was."""
    rng = np.random.default_rng([90, Hkv, N])
    D, T = 64, TYPES[kind]
    cache = as_cache(*random_cache(rng, 2, Hkv, 4, D, 4, 32))
    slots = i64(rng.permutation(8)[:N])
    want = [torch.empty((N, Hkv, D), dtype=T, device="cuda") for _ in range(2)]
    abg.kvq_get(cache, *want, slots=slots)
    for shape, parts in (((N, 2 * Hkv, D), lambda b: (b[:, 0::2], b[:, 1::2])),
                         ((N, 2 * Hkv + 1, D), lambda b: (b[:, 1::2], b[:, 0:2 * Hkv:2])),
                         ((N, 2 * Hkv + 1, D), lambda b: (b[:, Hkv + 1:], b[:, :Hkv])),
                         ((Hkv, N, 2, D), lambda b: (b[:, :, 0].transpose(0, 1), b[:, :, 1].transpose(0, 1))),
                         ((Hkv, 2, N, D), lambda b: (b[:, 1].transpose(0, 1), b[:, 0].transpose(0, 1))),
                         ((Hkv, N + 1, 3, D), lambda b: (b[:, :N, 2].transpose(0, 1), b[:, 1:, 0].transpose(0, 1)))):
        got, exp = (torch.full(shape, 7.0, dtype=T, device="cuda") for _ in range(2))
        abg.kvq_get(cache, *parts(got), slots=slots)
        for to, x in zip(parts(exp), want):
            to.copy_(x)
        assert torch.equal(got, exp), shape
    if N > 1:
        both = torch.zeros((N, 2 * Hkv, D), dtype=T, device="cuda")
        with pytest.raises(abg.AbgError, match="output overlaps"):
            abg.kvq_get(cache, both[:, :Hkv], both[:, Hkv - 1:2 * Hkv - 1], slots=slots)


# --------------------------------------------------------------- kvq_attn ----
def attn_case(seed, kind, bits, group, Hq, Hkv, D, page, lens, spans, words=None, gate=True, y32=False, tail=2, qscale=2.0):
    """Inputs (device) of one call: random pages, masks of random trees, NaN
    factors in every cache row past a request's length and in the unused pages,
    and NaN in the draft rows past the spans."""
    rng = np.random.default_rng([seed, D, page, bits, group])
    T = TYPES[kind]
    B, lens, spans = len(lens), np.array(lens), np.array(spans)
    words = words or max(1, -(-int(max(spans)) // 64))
    cu = np.concatenate([[0], np.cumsum(spans)])
    N = int(cu[-1]) + tail
    counts = -(-lens // page)
    pages, width = int(counts.sum()) + 2, int(max(1, counts.max()))
    order = rng.permutation(pages)
    table = rng.choice([-1, pages, 2**31 - 1, -2**31], (B, width))
    parts = random_cache(rng, pages, Hkv, page, D, bits, group)
    used = np.zeros((pages, page), bool)
    at = 0
    for b in range(B):
        table[b, :counts[b]] = order[at:at + counts[b]]
        at += counts[b]
        t = np.arange(lens[b])
        used[table[b, t // page], t % page] = True
    for p in (parts[1], parts[3]):
        p.transpose(0, 2, 1, 3, 4)[~used] = np.nan
    Kd, Vd = (rng.standard_normal((Hkv, N + 3, D)) for _ in range(2))
    Kd[:, cu[-1]:] = Vd[:, cu[-1]:] = np.nan
    parent = np.concatenate([parents(rng, spans), np.full(tail, -2, np.int32)])
    mask, _ = draft_ref.tree_plan(parent, lens, cu, words)
    t = lambda x: torch.from_numpy(x).to(T).cuda()  # noqa: E731
    return dict(q=t(qscale * rng.standard_normal((N, Hq, D))), cache=as_cache(*parts), table=i32(table), lens=i32(lens),
                cu=i32(cu), Kd=t(Kd), Vd=t(Vd), mask=i64(mask), max_span=int(max(1, min(max(spans), 64 * words))),
                gate=dev(rng.standard_normal((N, Hq, D)).astype(np.float32)) if gate else None,
                y=torch.full((N, Hq, D), 5.0, dtype=torch.float32 if y32 else T, device="cuda")), kind


def check_attn(c, kind, ysum=False):
    c = dict(c)
    if ysum:
        c["ysum"] = torch.full((c["y"].numel() // 64,), 5.0, device="cuda")
    abg.kvq_attn(**c)
    w = {k: None if c[k] is None else wide(c[k]) for k in ("q", "Kd", "Vd", "gate")}
    Kw, Kp, Vw, Vp = arrays(c["cache"])
    bits = 32 * Kw.shape[-1] // w["q"].shape[2]
    (K, Kmag), (V, Vmag) = ref.values(Kw, Kp, bits), ref.values(Vw, Vp, bits)
    seen = bits_of(c["mask"])
    plan = host(c["table"]), host(c["lens"]), host(c["cu"])
    want, _ = draft_ref.tree_attn(w["q"], K, V, *plan, w["Kd"], w["Vd"], seen, w["gate"])
    # of each row the largest |scale| code + |bias| of V, and sum of |q_i| (|scale| code + |bias|) / sqrt(D)
    # (NaN left out: a result that it reaches is NaN, whatever the bound)
    Kmag, Vmag = np.nan_to_num(Kmag), np.nan_to_num(Vmag)
    _, terms = draft_ref.tree_attn(np.abs(w["q"]), Kmag, Vmag, *plan, np.abs(w["Kd"]), np.abs(w["Vd"]), seen)
    got = wide(c["y"])
    cu, cap = plan[2], seen.shape[1]
    written = np.zeros(len(got), bool)
    for b in range(len(cu) - 1):
        written[cu[b]:min(cu[b + 1], cu[b] + cap)] = True
    assert np.all(got[~written] == 5.0)
    # f32 steps: a score's D + 8 sums of its magnitudes (the tensor cores may cut
    # them off: two roundings each; an error moves a weight by as much, numerator
    # and denominator), q to 22 bits or 2^-34 of its row's largest; the weight
    # itself and its place in the sum, the joins of at most 600 pieces, the gate
    D, n = w["q"].shape[2], int(plan[1].max()) + cap
    top, mag = terms[..., :1], terms[..., 1:]
    bound = U32 * top * (2 * (2 * (D + 8) + (4 if kind == "f32" else 0)) * mag + 4 * (64 + n / 16 + 600))
    if kind == "f32":
        with np.errstate(invalid="ignore"):
            bound += 2 * 2.0**-34 * np.abs(w["q"]).max(2, keepdims=True) * np.nanmax(Kmag, initial=0) * np.sqrt(D) * top
    # the weights that meet the codes: 11 or 22 bits, or 2^-38 of the largest scale of V
    bound += top * ((2.0**-11 if kind == "bf16" else 2.0**-22) + n * 2.0**-38) * 1.01
    if c["y"].dtype != torch.float32:
        bound = bound + UNIT[kind] * np.abs(want) * 1.02 + 2.0**-25  # y's own
    err = np.abs(got - want)
    ok = (err <= bound) | (np.isnan(got) & np.isnan(want)) | (got == want)
    assert ok[written].all(), (np.argwhere(~ok & written[:, None, None])[:5], np.nanmax(err), np.nanmax(err[written] / bound[written]))
    if ysum:
        y = got.reshape(len(got), -1, 64)
        s = host(c["ysum"]).reshape(y.shape[:2]).astype(np.float64)
        assert np.all(np.abs(s - y.sum(2))[written] <= 64 * U32 * np.abs(y).sum(2)[written] + 1e-30)
        assert np.all(s[~written] == 5.0)
    return got, want


FORMATS = [(4, 64), (4, 32), (8, 64), (8, 32)]
ATTN = [  # Hq, Hkv, D, page, lens, spans
    (8, 2, 256, 64, [2047], [1]),
    (4, 4, 64, 16, [0], [1]),
    (4, 2, 128, 16, [1], [1]),
    (6, 3, 64, 7, [64, 0, 63, 65, 300], [1, 3, 0, 17, 2]),
    (16, 4, 128, 16, [127, 128, 129, 1000], [24, 7, 64, 1]),
    (16, 2, 256, 32, [513, 40], [8, 8]),
    (3, 1, 128, 1, [77, 5], [30, 64]),
    (8, 1, 64, 1000, [999, 1001, 2000], [5, 63, 33]),
    (5, 5, 256, 48, [191, 95], [64, 10]),
    (8, 2, 128, 128, [4000], [1]),
    (2, 2, 64, 100, [20000], [2]),
    (16, 1, 128, 24, [0, 0, 700], [1, 2, 3]),
    (12, 2, 128, 16, [15, 16, 17, 31, 32, 33, 255, 256, 257], [1] * 9),
]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,spans", ATTN)
def test_kvq_attn(kind, bits, group, Hq, Hkv, D, page, lens, spans):
    check_attn(*attn_case(1, kind, bits, group, Hq, Hkv, D, page, lens, spans, gate=D != 128))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bits,group", FORMATS)
@pytest.mark.parametrize("spans", [[65, 128], [150, 1, 192], [256, 30]])
def test_kvq_attn_spans_past_one_mask_word(kind, bits, group, spans):
    check_attn(*attn_case(2, kind, bits, group, 8, 2, 128, 16, [200, 33, 150][:len(spans)], spans))
    check_attn(*attn_case(3, kind, bits, group, 3, 1, 256, 16, [130, 1, 0][:len(spans)], spans, gate=False))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", FORMATS)
def test_kvq_attn_f32_result_and_group_sums(kind, bits, group):
    check_attn(*attn_case(4, kind, bits, group, 8, 2, 256, 16, [700, 15], [8, 3], y32=True), ysum=True)
    check_attn(*attn_case(5, kind, bits, group, 4, 2, 64, 16, [9000], [4], y32=True), ysum=True)
    check_attn(*attn_case(6, kind, bits, group, 16, 4, 128, 16, [300, 100], [40, 20], y32=True, gate=False), ysum=True)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", FORMATS)
def test_kvq_attn_many_ragged_requests(kind, bits, group):
    rng = np.random.default_rng(8)
    lens, spans = rng.integers(0, 700, 300), rng.integers(0, 6, 300)
    check_attn(*attn_case(7, kind, bits, group, 4, 2, 64, 16, lens, spans))
    check_attn(*attn_case(8, kind, bits, group, 8, 1, 128, 16, lens[:170], np.minimum(spans[:170], 1)))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_kvq_attn_rows_that_see_nothing_are_zero(kind, bits, group):
    c, k = attn_case(9, kind, bits, group, 4, 2, 128, 16, [0, 40, 0], [6, 5, 70], gate=False)
    mask = host(c["mask"]).copy()
    mask[[2, 3, 7, 12, 60]] = 0
    c["mask"] = i64(mask)
    got, _ = check_attn(c, k)
    assert np.all(got[[2, 3, 12, 60]] == 0) and np.all(np.abs(got[7]).max(1) > 0)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_kvq_attn_bad_pages_read_as_zeros(kind):
    for bits, group in FORMATS:
        c, k = attn_case(12, kind, bits, group, 4, 2, 64, 16, [200, 100], [3, 3])
        table = host(c["table"]).copy()
        table[0, 2], table[1, 0], table[0, 5] = -7, 2**31 - 1, -2**31
        check_attn(dict(c, table=i32(table)), k)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 256])
def test_kvq_attn_nan_stays_where_it_is_seen(kind, D):
    """NaN and infinities in K and V of one draft reach the drafts that see it; a
    NaN row of the cache its request, in V the group's columns; a NaN or a huge q
    its own row."""
    c, k = attn_case(10, kind, 4, 32, 6, 3, D, 16, [50, 40], [40, 90], gate=False)
    bits = bits_of(c["mask"])
    Kd, Vd, q = c["Kd"].clone(), c["Vd"].clone(), c["q"].clone()
    bad = {5: (float("nan"), 1.0), 17: (1.0, float("nan")), 30: (1.0, float("inf")), 110: (1.0, float("-inf"))}
    for n, (fk, fv) in bad.items():
        Kd[:, n, 3] *= fk
        Vd[:, n, 7] *= fv
    q[2, 1, 9], q[3, 4, 60] = float("nan"), float("inf")
    if kind != "f16":
        q[20, 0, 1] = 2.0**101
    y = torch.zeros_like(c["y"])
    abg.kvq_attn(**dict(c, q=q, Kd=Kd, Vd=Vd, y=y))
    got = wide(y)
    for lo, hi in ((0, 40), (40, 130)):
        sees = np.array([[lo <= n < hi and bits[t, n - lo] for n in bad] for t in range(lo, hi)])
        own = np.zeros((hi - lo, 6), bool)
        if lo == 0:
            own[2, 1] = own[3, 4] = True
            own[20, 0] = kind != "f16"
        assert np.isnan(got[lo:hi][own]).all()
        plain = ~sees.any(1)[:, None] & ~own
        assert np.isfinite(got[lo:hi][plain]).all()
        assert np.isnan(got[lo:hi][sees[:, 0]]).all()
        only = ((sees[:, 1] | sees[:, 2] | sees[:, 3]) & ~sees[:, 0])[:, None] & ~own
        assert not np.isfinite(got[lo:hi][only][:, 7]).any() and np.isfinite(got[lo:hi][only][:, 8:]).all()
    # request 1's cached rows: V of head 2, group 1; then K of head 1
    Kw, Kp, Vw, Vp = arrays(c["cache"])
    page = host(c["table"])[1, 1]
    Vp = Vp.copy()
    Vp[page, 2, 5, 1] = np.nan
    got, _ = check_attn(dict(c, cache=as_cache(Kw, Kp, Vw, Vp), y=c["y"].clone()), k)
    assert np.isnan(got[40:130, 4:, 32:64]).all() and np.isfinite(got[40:130, 4:, :32]).all() and np.isfinite(got[:40]).all()
    Kp = Kp.copy()
    Kp[page, 1, 15, 0, 1] = np.nan
    abg.kvq_attn(**dict(c, cache=as_cache(Kw, Kp, Vw, arrays(c["cache"])[3])))
    got = wide(c["y"])
    assert np.isnan(got[40:130, 2:4]).all() and np.isfinite(got[40:130, :2]).all() and np.isfinite(got[:40]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,top,bad", [(600, 5, 40), (600, 40, 5), (600, 5, 590), (20000, 5, 19990), (20000, 19990, 5),
                                            (20000, 12000, 5)])
def test_kvq_attn_nan_far_below_the_largest_score_stays(kind, tokens, top, bad):
    """A NaN in a row that another warp, block or piece outweighs by 2^800."""
    c, k = attn_case(14, kind, 4, 32, 4, 2, 128, 16, [tokens], [2], gate=False)
    Kw, Kp, Vw, Vp = (a.copy() for a in arrays(c["cache"]))

    def at(t):
        return host(c["table"])[0][t // 16], slice(None), t % 16

    Kp[(*at(np.arange(tokens)), 0, slice(None))] = 0.0
    Kp[(*at(top), 0, 1)] = 40.0
    q = c["q"].clone()
    q[..., :32] = 5.0
    Vp[at(bad)[0], 1, at(bad)[2], 2, 0] = np.nan
    y = torch.zeros_like(c["y"])
    abg.kvq_attn(**dict(c, cache=as_cache(Kw, Kp, Vw, Vp), q=q, y=y))
    got = wide(y)[:2]
    nan = np.zeros(got.shape, bool)
    nan[:, 2:, 64:96] = True
    assert np.array_equal(np.isnan(got), nan)
    Kp[at(bad)[0], 0, at(bad)[2], 3, 1] = np.nan
    abg.kvq_attn(**dict(c, cache=as_cache(Kw, Kp, Vw, Vp), q=q, y=y))
    nan[:, :2] = True
    assert np.array_equal(np.isnan(wide(y)[:2]), nan)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", [(4, 32), (8, 64)])
def test_kvq_attn_scores_far_apart_and_scales_of_all_sizes(kind, bits, group):
    """Scores that grow along the sequence (every block raises the maximum) and
    that fall, over +-200; scales of V from f16's smallest to its large ones, so
    that the weights' power of two grows along the way."""
    for sign in (1.0, -1.0):
        c, k = attn_case(11, kind, bits, group, 4, 2, 128, 16, [1500], [6], gate=False)
        Kw, Kp, Vw, Vp = (a.copy() for a in arrays(c["cache"]))
        t = np.arange(1500)
        at = host(c["table"])[0][t // 16], slice(None), t % 16
        ramp = np.linspace(-1, 1, 1500) * sign
        Kp[(*at, 0, 1)] = (ramp * 14 * 8 / 32)[:, None]  # the bias of the first group
        q = c["q"].clone()
        q[..., :32] = 5.0
        if group == 64:
            q[..., 32:64] = 0.0
        check_attn(dict(c, cache=as_cache(Kw, Kp, Vw, Vp), q=q, y=c["y"].clone()), k)
        Vp[(*at, slice(None), 0)] *= (2.0 ** np.linspace(-18, 12, 1500))[::int(sign)][:, None, None]
        check_attn(dict(c, cache=as_cache(Kw, Kp, Vw, Vp), q=c["q"] * 0.25, y=c["y"].clone()), k)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_kvq_attn_negative_and_large_factors(kind):
    """A cache that another program made: scales of either sign, codes that fill
    their words, rows of q of very different sizes."""
    rng = np.random.default_rng(40)
    for bits, group in FORMATS:
        c, k = attn_case(14, kind, bits, group, 8, 2, 128, 16, [333, 90], [2, 5])
        Kw, Kp, Vw, Vp = (a.copy() for a in arrays(c["cache"]))
        Kw[:], Vw[:] = rng.integers(0, 2**32, Kw.shape, dtype=np.uint32), rng.integers(0, 2**32, Vw.shape, dtype=np.uint32)
        for p in (Kp, Vp):
            p[..., 0] *= rng.choice([-1.0, 1.0], p.shape[:-1]).astype(np.float16)
        q = c["q"] * torch.from_numpy(2.0 ** rng.integers(-14, 2, (len(c["q"]), 8, 1))).to(c["q"].dtype).cuda()
        check_attn(dict(c, q=q, cache=as_cache(Kw, Kp, Vw, Vp)), k)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tall", [[(0, 25.4)], [(70000, 20.7)], [(131071, 25.4)], [(5, 25.4), (6, 18.0)]])
def test_kvq_attn_many_weights_far_below_the_largest(kind, tall):
    """131072 tokens of one score under one or two that are far above (log2 of the
    weights' ratio given): the small weights together count.  V is 1 (scale 1, code
    1) where the score is small and 0 where it is large; requests that share the
    cache, so many that most of them are not cut."""
    n, page, B, D = 131072, 128, 320, 64
    pairs = [np.zeros((n // page, 1, page, 1, 2), np.float16) for _ in range(2)]
    words = [np.zeros((n // page, 1, page, 8), np.uint32) for _ in range(2)]
    words[1][:] = 0x11111111
    pairs[1][..., 0] = 1.0
    q = np.zeros((B, 1, D), np.float32)
    q[..., 0] = 16.0
    for t, lg in tall:
        pairs[0][t // page, 0, t % page, 0, 1] = lg * np.log(2) * np.sqrt(D) / 16.0  # K is the bias; q sums to 16
        words[1][t // page, 0, t % page] = 0
    s = pairs[0][..., 0, 1].astype(np.float64).ravel() * 16 / np.sqrt(D)
    w = np.exp(s - s.max())
    want = (w * (words[1][..., 0] > 0).ravel()).sum() / w.sum()
    y = torch.empty((B, 1, D), device="cuda")
    draft = torch.zeros((1, B, D), dtype=TYPES[kind], device="cuda")
    abg.kvq_attn(torch.from_numpy(q).to(TYPES[kind]).cuda(), as_cache(words[0], pairs[0], words[1], pairs[1]),
                 i32(np.arange(n // page)[None].repeat(B, 0)), i32([n] * B), i32(np.arange(B + 1)), draft, draft,
                 i64(np.zeros((B, 1))), y)
    # the weights' rounding; in f32, a score's and a weight's few roundings, sums of
    # 16 at a time that may be cut off (two roundings each), joins
    bound = (2.0**-11 if kind == "bf16" else 2.0**-22) * 1.01 * want + n * 2.0**-38 + want * U32 * (2 * n / 16 + 600)
    assert np.abs(host(y) - want).max() <= bound, (host(y).min(), host(y).max(), want, bound)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", FORMATS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_kvq_attn_scores_whose_rounding_moves_a_weight(kind, bits, group, sign):
    """Rows of q up to 2^95, so that a score's last bit is worth many powers of two:
    the largest score has all the weight, and rows of moderate scores beside them
    are as exact as alone.  K is a bias of whole numbers, each once, in its first
    group, where q is constant, and q is 0 elsewhere."""
    c, _ = attn_case(15, kind, bits, group, 4, 2, 128, 16, [700], [6], gate=False, y32=True, tail=0)
    rng = np.random.default_rng([80, bits, group])
    Kw, Kp, Vw, Vp = (a.copy() for a in arrays(c["cache"]))
    t = np.arange(700)
    at = host(c["table"])[0][t // 16], slice(None), t % 16
    bias = sign * (1 + rng.permutation(1500)[:700])
    Kp[(*at, 0, 0)], Kp[(*at, 0, 1)] = 0.0, bias[:, None]
    top = np.array([-6, 10, 12, 13, 14, 11] if kind == "f16" else [-6, 16, 18, 23, 30, 95])
    q = np.zeros((6, 4, 128))
    q[..., :group] = (rng.uniform(1, 2, (6, 4)) * 2.0 ** top[:, None])[..., None]
    Kd = np.zeros((2, 9, 128))
    Kd[:, :6, :group] = 3008.0 if sign > 0 else -0.25  # above all of the cache's
    c.update(q=torch.from_numpy(q).to(TYPES[kind]).cuda(), Kd=torch.from_numpy(Kd).to(TYPES[kind]).cuda(),
             cache=as_cache(Kw, Kp, Vw, Vp))
    (K, _), (V, Vmag) = ref.values(Kw, Kp, bits), ref.values(Vw, Vp, bits)
    Vd, far = wide(c["Vd"]), top > 0
    for own in (False, True):
        mask = np.where(own, 1 << np.arange(6), 0)[:, None]
        y = torch.full_like(c["y"], 5.0)
        abg.kvq_attn(**dict(c, mask=i64(mask), y=y))
        got = wide(y).reshape(6, 2, 2, 128)  # of two query heads a cached head
        if own:
            want, mag = Vd[:, :6].swapaxes(0, 1)[:, :, None], np.abs(Vd[:, :6]).swapaxes(0, 1)[:, :, None]
        else:
            w = int(np.argmax(bias))
            want, mag = (x[host(c["table"])[0][w // 16], :, w % 16][None, :, None] for x in (V, Vmag))
        # one weight that is not 0: rounded, as its scale times it and the products, to 11 or 22 bits and cut off
        # at 2^-17 or 2^-23 (twice each), and some sixteen steps in f32 from there to the quotient
        bound = mag * (2.0**-11 + 2 * 2.0**-17 if kind == "bf16" else 2.0**-22 + 2 * 2.0**-23) + mag * 16 * U32
        err = np.abs(got - want)
        assert (err <= bound)[far].all(), (own, top, np.nanmax(err / mag, axis=(1, 2, 3)), np.isnan(got).any(axis=(1, 2, 3)))
        if not own:
            # the row of moderate scores: f32 steps of a score's magnitude (as check_attn's)
            exact, terms = (draft_ref.tree_attn(f(wide(c["q"])), k, v, host(c["table"]), host(c["lens"]), host(c["cu"]),
                                                f(wide(c["Kd"])), f(Vd), bits_of(i64(mask)))[i]
                            for i, f, k, v in ((0, np.array, K, V), (1, np.abs, np.nan_to_num(ref.values(Kw, Kp, bits)[1]),
                                                                     np.nan_to_num(Vmag))))
            high, mags = terms[..., :1], terms[..., 1:]
            room = high * (U32 * (2 * (2 * (128 + 8) + 4) * mags + 4 * (64 + 700 / 16 + 600)) +
                           ((2.0**-11 if kind == "bf16" else 2.0**-22) + 700 * 2.0**-38) * 1.01)
            assert (np.abs(wide(y) - exact) <= room)[~far].all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [-24, -20, -16, -14])
@pytest.mark.parametrize("tall", [[(0, 28.5)], [(5, 30.0), (6, 18.0)]])
def test_kvq_attn_many_small_weights_and_small_scales(kind, scale, tall):
    """test_kvq_attn_many_weights_far_below_the_largest with V's scale a power of two
    down to f16's smallest: the same result times it."""
    n, page, B, D = 131072, 128, 320, 64
    pairs = [np.zeros((n // page, 1, page, 1, 2), np.float16) for _ in range(2)]
    words = [np.zeros((n // page, 1, page, 8), np.uint32) for _ in range(2)]
    words[1][:] = 0x11111111
    pairs[1][..., 0] = 2.0**scale
    q = np.zeros((B, 1, D), np.float32)
    q[..., 0] = 16.0
    for t, lg in tall:
        pairs[0][t // page, 0, t % page, 0, 1] = lg * np.log(2) * np.sqrt(D) / 16.0  # K is the bias; q sums to 16
        words[1][t // page, 0, t % page] = 0
    s = pairs[0][..., 0, 1].astype(np.float64).ravel() * 16 / np.sqrt(D)
    w = np.exp(s - s.max())
    want = (w * (words[1][..., 0] > 0).ravel()).sum() / w.sum()
    y = torch.empty((B, 1, D), device="cuda")
    draft = torch.zeros((1, B, D), dtype=TYPES[kind], device="cuda")
    abg.kvq_attn(torch.from_numpy(q).to(TYPES[kind]).cuda(), as_cache(words[0], pairs[0], words[1], pairs[1]),
                 i32(np.arange(n // page)[None].repeat(B, 0)), i32([n] * B), i32(np.arange(B + 1)), draft, draft,
                 i64(np.zeros((B, 1))), y)
    # as there, all of it in units of the scale
    bound = (2.0**-11 if kind == "bf16" else 2.0**-22) * 1.01 * want + n * 2.0**-38 + want * U32 * (2 * n / 16 + 600)
    got = host(y).astype(np.float64) * 2.0**-scale
    assert np.abs(got - want).max() <= bound, (got.min(), got.max(), want, bound)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_kvq_attn_large_draft_keys_under_small_queries(kind, D):
    """Drafts' K of 2^116 with q of 2^-80, whose products would pass f32's range with q
    brought up to f16's, and the other way round: finite results."""
    c, k = attn_case(16, kind, 4, 32, 4, 2, D, 16, [100, 0], [5, 9], gate=False)
    for q, e in ((2.0**-80, 2.0**116), (2.0**-115, 2.0**115), (2.0**60, 2.0**-60)):
        check_attn(dict(c, q=c["q"] * q, Kd=c["Kd"] * e, y=c["y"].clone(), lens=i32([100 if q < 1 else 0, 0])), k)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tiles", [16, 17, 18, 40, 120])
def test_kvq_attn_infinity_far_below_the_largest_score_stays(kind, tiles):
    """An infinite value of a draft, in the unit's last piece, that another piece
    outweighs by 2^800: infinite or (infinity times 0) NaN, whichever of a row's warps
    joins its piece, and never a number."""
    tokens = 128 * tiles
    c, k = attn_case(17, kind, 4, 32, 4, 2, 128, 16, [tokens], [1], gate=False, tail=0)
    Kw, Kp, Vw, Vp = (a.copy() for a in arrays(c["cache"]))
    q, Kd, Vd = c["q"].clone(), c["Kd"].clone(), c["Vd"].clone()
    q[..., :32], Kd[:], c["mask"] = 5.0, 0.0, i64([[1]])
    Vd[0, 0, 70], Vd[1, 0, 5] = float("inf"), float("-inf")
    want = np.zeros((1, 4, 128), bool)
    want[:, :2, 70] = want[:, 2:, 5] = True
    every = np.arange(tokens)
    Kp[host(c["table"])[0][every // 16], :, every % 16, 0] = 0.0
    for top in (5, 700, 1300, tokens - 5):
        p = Kp.copy()
        p[host(c["table"])[0][top // 16], :, top % 16, 0, 1] = 40.0
        y = torch.zeros_like(c["y"])
        abg.kvq_attn(**dict(c, cache=as_cache(Kw, p, Vw, Vp), q=q, Kd=Kd, Vd=Vd, y=y))
        assert np.array_equal(~np.isfinite(wide(y)), want), top


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_kvq_attn_is_the_same_on_every_run_and_on_other_streams(kind):
    c, k = attn_case(13, kind, 4, 64, 8, 2, 128, 16, [5000, 70, 900], [4, 3, 1])
    abg.kvq_attn(**c)
    first = c["y"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    ws = [torch.empty(abg.kvq_attn_workspace(c["q"], c["cache"], c["max_span"]), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    for i in range(20):
        y = torch.empty_like(first)
        s = side if i % 2 else torch.cuda.current_stream()
        abg.kvq_attn(**dict(c, y=y), ws=ws[i % 2], stream=s)
        outs.append(y)
    torch.cuda.synchronize()
    written = int(host(c["cu"])[-1])
    for y in outs:
        assert torch.equal(y[:written], first[:written])


# ------------------------------------------------- together, and captured ----
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", FORMATS)
def test_put_attend_and_read_back_is_attention_over_the_rows_read_back(kind, bits, group):
    """Rows put through a plan's slots, then attended to, against tree_attn over
    the rows that kvq_get gives (both within their bounds of the exact value)."""
    rng = np.random.default_rng([50, bits, group])
    T, B, Hq, Hkv, D, page, width = TYPES[kind], 3, 8, 2, 128, 16, 40
    lens = np.array([300, 17, 555])
    N = int(lens.sum())
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    ring, table = i32(rng.permutation(60)), i32(np.zeros((B, width)))
    slots, pos = i64(np.zeros(N)), i32(np.zeros(N))
    out = i32(np.zeros(B)), i32(np.zeros(B)), i64([0, 0]), i32([0, 0])
    abg.page_plan(i32([0] * B), i32(lens), cu, i32([0] * B), i64([0, 60]), ring, table, page, slots, pos, *out)
    cache = abg.kvq_cache(60, Hkv, page, D, bits, group)
    kv = torch.randn((N, 2 * Hkv, D), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    abg.kvq_put(kv[:, :Hkv], kv[:, Hkv:], cache, slots=slots)
    # the values, in a cache of their own
    every = i64(np.arange(60 * page))
    plain = [torch.empty((60 * page, Hkv, D), device="cuda") for _ in range(2)]
    abg.kvq_get(cache, *plain, slots=every)
    plain = [x.view(60, page, Hkv, D).transpose(1, 2).contiguous() for x in plain]
    q = torch.randn((B, Hq, D), device="cuda").to(T)
    Kd, Vd = (torch.randn((Hkv, B, D), device="cuda").to(T) for _ in range(2))
    mask, one = i64(np.ones((B, 1))), i32(np.arange(B + 1))
    y, z = (torch.empty((B, Hq, D), device="cuda") for _ in range(2))
    abg.kvq_attn(q, cache, table, out[0], one, Kd, Vd, mask, y, max_span=1)
    abg.tree_attn(q.float(), *plain, table, out[0], one, Kd.float(), Vd.float(), mask, z, max_span=1)
    top = float(max(plain[1].abs().max(), Vd.abs().max())) * 2
    mag = float((q.float().abs().sum(2).max() * max(plain[0].abs().max(), Kd.abs().max())) / np.sqrt(D)) * 2
    bound = top * (2.0**-11 if kind == "bf16" else 2.0**-22) + 2 * U32 * top * (4 * (D + 10) * mag + 4 * (64 + 600 + 40))
    assert float((y - z).abs().max()) <= bound


def test_calls_record_into_a_cuda_graph():
    c, _ = attn_case(30, "bf16", 4, 64, 8, 2, 128, 16, [300, 90], [6, 4], tail=0)
    ws = torch.empty(abg.kvq_attn_workspace(c["q"], c["cache"], c["max_span"]), dtype=torch.uint8, device="cuda")
    k, v = (torch.randn((2, 2, 128), device="cuda") for _ in range(2))
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    pages = host(c["table"])
    slots = i64([pages[0, 18] * 16 + 11, pages[1, 5] * 16 + 9])  # the last cached token of each

    def step():
        abg.kvq_put(k, v, c["cache"], slots=slots)
        abg.kvq_attn(**c, ws=ws)
        abg.kvq_get(c["cache"], ko, vo, slots=slots)

    step()
    want = c["y"].clone(), ko.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c["y"].fill_(5.0), ko.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c["y"], want[0]) and torch.equal(ko, want[1])
    k.mul_(-2.0)  # new rows: the replay's results are theirs
    g.replay()
    got = c["y"].clone(), ko.clone()
    step()
    assert torch.equal(got[0], c["y"]) and torch.equal(got[1], ko) and not torch.equal(got[0], want[0])


# ------------------------------------------------------------ far offsets ----
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_pages_past_two_to_the_32_columns(bits, group):
    """More than 2^32 columns and, in 8 bits, bytes; rows put into the last pages
    are found there."""
    Hkv, page, D, pages = 4, 64, 256, 70000
    assert pages * Hkv * page * D > 2**32
    shape = (pages, Hkv, page)
    cache = abg.KvqCache(*(torch.empty((*shape, *s), dtype=t, device="cuda") for s, t in (
        ((D * bits // 32,), torch.int32), ((D // group, 2), torch.float16)) * 2))
    n = 100
    table = np.array([[pages - 1, pages - 2]])
    k, v = (torch.randn((n, Hkv, D), device="cuda") for _ in range(2))
    t = np.arange(n)
    slots = i64(table[0, t // page].astype(np.int64) * page + t % page)
    abg.kvq_put(k, v, cache, slots=slots)
    words, pairs = ref.quantise(host(k), bits, group)
    same_bits(host(cache.Kc[-1]).view(np.uint32).transpose(1, 0, 2), words[:page])
    same_bits(host(cache.Ks[-2])[:, :n - page].transpose(1, 0, 2, 3), pairs[page:])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    abg.kvq_get(cache, ko, vo, slots=slots)
    assert np.array_equal(host(ko), ref.values(words, pairs, bits)[0].astype(np.float32))
    c, _ = attn_case(50, "bf16", bits, group, 8, 4, D, page, [n], [5], gate=False)
    c.update(cache=cache, table=i32(table))
    abg.kvq_attn(**c)
    far = c["y"].clone()
    c.update(cache=abg.KvqCache(*(x[-2:].clone() for x in cache)), table=i32([[1, 0]]))
    abg.kvq_attn(**c)
    assert torch.equal(far[:5], c["y"][:5])
    check_attn(c, "bf16")


def test_a_cache_without_pages_and_requests_without_tokens():
    """No page at all, tables of no width, empty spans: only the drafts count; a
    row that has none is not written."""
    for kind in ("bf16", "f32"):
        c, k = attn_case(60, kind, 4, 64, 4, 2, 64, 16, [0, 0, 0], [2, 0, 1], gate=False)
        want, _ = check_attn(dict(c, y=c["y"].clone()), k)
        empty = abg.kvq_cache(0, 2, 16, 64)
        for table in (c["table"], i32(np.zeros((3, 0)))):
            y = torch.full_like(c["y"], 5.0)
            abg.kvq_attn(**dict(c, cache=empty, table=table, lens=i32([40, 7, 2**31 - 1]) if table.numel() == 0 else c["lens"], y=y))
            assert np.array_equal(wide(y), want)
    rows = torch.ones((3, 2, 64), device="cuda")
    abg.kvq_put(rows, rows, empty)
    abg.kvq_get(empty, rows, None, slots=i64([0, 1, 2]))
    assert not rows.any()
    abg.kvq_put(rows[:0], rows[:0], empty)
    abg.kvq_get(empty, rows[:0], None)


def test_lengths_that_are_out_of_range():
    """A negative length is 0; one past the table's width ends at its last token."""
    c, k = attn_case(61, "bf16", 4, 64, 8, 2, 128, 16, [64, 32, 48], [1, 2, 1], gate=False)
    check_attn(dict(c, lens=i32([-5, 2**31 - 1, 48]), table=i32(np.where(host(c["table"]) < 0, -1, host(c["table"])))), k)


@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_rows_between_other_rows(bits, group):
    """Sources and results inside wider rows, heads before rows, one head alone."""
    rng = np.random.default_rng([70, bits])
    N, Hkv, D = 19, 3, 128
    wide_rows = dev(rng.standard_normal((N, 3 * Hkv + 2, D + 16)).astype(np.float32))
    k, v = wide_rows[:, 1:1 + 2 * Hkv:2, :D], wide_rows[:, 2 * Hkv:3 * Hkv, 16:]
    cache = abg.kvq_cache(2, Hkv, 13, D, bits, group)
    abg.kvq_put(k, v, cache)
    for i, x in ((0, k), (2, v)):
        words, pairs = ref.quantise(host(x.contiguous()), bits, group)
        got = [a.transpose(0, 2, 1, *range(3, a.ndim)).reshape(26, Hkv, *a.shape[3:])[:N] for a in arrays(cache)[i:i + 2]]
        same_bits(got[0], words)
        same_bits(got[1], pairs)
    ko, vo = torch.empty((N, Hkv, D), device="cuda"), torch.empty((N, Hkv, D), device="cuda")
    abg.kvq_get(cache, ko, vo)
    out = torch.zeros_like(wide_rows)
    abg.kvq_get(cache, out[:, 1:1 + 2 * Hkv:2, :D], None)
    abg.kvq_get(cache, None, out[:, 2 * Hkv:3 * Hkv, 16:])
    assert torch.equal(out[:, 1:1 + 2 * Hkv:2, :D], ko) and torch.equal(out[:, 2 * Hkv:3 * Hkv, 16:], vo)
    out[:, 1:1 + 2 * Hkv:2, :D] = 0
    out[:, 2 * Hkv:3 * Hkv, 16:] = 0
    assert not out.any()


def test_early_start_off_gives_the_same_bits(tmp_path):
    """ABG_PDL=0 in a process of its own: plain stream order, the same results."""
    import os
    import subprocess
    import sys
    prog = tmp_path / "run.py"
    prog.write_text(
        "import sys, torch\n"
        f"sys.path[:0] = {[os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__))]!r}\n"
        "import test_gpu_9_kvq as t\n"
        "out = []\n"
        "for kind, bits in (('f32', 4), ('bf16', 8), ('f16', 4)):\n"
        "    c, _ = t.attn_case(60, kind, bits, 64, 8, 2, 128, 16, [900, 40], [9, 30], tail=0)\n"
        "    k = torch.arange(2 * 2 * 128, device='cuda').view(2, 2, 128).float().sin()\n"
        "    for i in range(3):\n"
        "        t.abg.kvq_put(k * (i + 1), k, c['cache'], slots=t.i64([3, 18]))\n"
        "        t.abg.kvq_attn(**c)\n"
        "    ko = torch.empty_like(k)\n"
        "    t.abg.kvq_get(c['cache'], ko, None, slots=t.i64([3, 18]))\n"
        "    out += [c['y'].cpu(), ko.cpu()]\n"
        "torch.save(out, sys.argv[1])\n")
    got = []
    for v in ("0", "1"):
        path = tmp_path / v
        env = dict(os.environ, ABG_PDL=v)
        subprocess.run([sys.executable, str(prog), str(path)], check=True, env=env, timeout=120)
        got.append(torch.load(path))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_first_call_inside_a_capture():
    """A process whose first call of each kernel is recorded: nothing that a call
    sets up once is a stream operation."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([sys.executable, "-c",
                    "import sys, torch\n"
                    f"sys.path[:0] = {[os.path.dirname(here), here]!r}\n"
                    "import test_gpu_9_kvq as t\n"
                    "c, k = t.attn_case(30, 'bf16', 8, 32, 8, 2, 64, 16, [300, 90], [6, 4], tail=0)\n"
                    "ws = torch.empty(t.abg.kvq_attn_workspace(c['q'], c['cache'], c['max_span']), dtype=torch.uint8, device='cuda')\n"
                    "ko = torch.empty((2, 2, 64), device='cuda')\n"
                    "g = torch.cuda.CUDAGraph()\n"
                    "with torch.cuda.graph(g):\n"
                    "    t.abg.kvq_attn(**c, ws=ws)\n"
                    "    t.abg.kvq_get(c['cache'], ko, None)\n"
                    "g.replay()\n"
                    "y, r = c['y'].clone(), ko.clone()\n"
                    "t.check_attn(c, k)\n"
                    "t.abg.kvq_get(c['cache'], ko, None)\n"
                    "assert torch.equal(y, c['y']) and torch.equal(r.nan_to_num(7.0), ko.nan_to_num(7.0))\n"],
                   check=True, timeout=120)


# --------------------------------------------------------------- refusals ----
def test_binding_refuses_wrong_tensors_on_the_device():
    c, _ = attn_case(40, "bf16", 4, 64, 4, 2, 64, 16, [20], [3], tail=0)
    ws = torch.empty(abg.kvq_attn_workspace(c["q"], c["cache"], c["max_span"]), dtype=torch.uint8, device="cuda")
    cache = c["cache"]
    for change, words in ((dict(q=c["q"].transpose(0, 1)), "q must be"), (dict(q=c["q"][:, :, :33]), "rows are not of 33"),
                          (dict(Kd=c["Kd"].float()), "Kd must be a contiguous torch.bfloat16"),
                          (dict(lens=c["lens"].long()), "lens must be a contiguous torch.int32"),
                          (dict(mask=c["mask"][:2]), "mask must be"), (dict(y=c["y"].int()), "y must be float32"),
                          (dict(ws=ws.int()), "ws must be a contiguous torch.uint8"), (dict(cache=list(cache)), "tuple"),
                          (dict(cache=cache[:3]), "tuple"), (dict(cache=cache._replace(Ks=cache.Ks[:1])), "words"),
                          (dict(cache=cache._replace(Ks=cache.Ks.float())), "Ks must be a contiguous torch.float16"),
                          (dict(cache=cache._replace(Vc=cache.Vc.transpose(0, 1).contiguous().transpose(0, 1))), "Vc must be")):
        with pytest.raises(ValueError, match=words):
            abg.kvq_attn(**{**c, "ws": ws, **change})
    with pytest.raises(abg.AbgError, match="bad shape"):
        abg.kvq_attn(**dict(c, ws=ws[:64]))
    with pytest.raises(abg.AbgError, match="output overlaps"):
        abg.kvq_attn(**dict(c, y=c["q"], ws=ws))
    wide_words = torch.zeros((2, 2, 16, 32), dtype=torch.int32, device="cuda")  # 16 bits a column
    with pytest.raises(abg.AbgError, match="invalid argument"):
        abg.kvq_attn(**dict(c, cache=abg.KvqCache(wide_words, torch.zeros((2, 2, 16, 1, 2), dtype=torch.float16, device="cuda"),
                                                  wide_words, torch.zeros((2, 2, 16, 1, 2), dtype=torch.float16, device="cuda")), ws=ws))
    k = torch.zeros((3, 2, 128), device="cuda")
    cache = abg.kvq_cache(1, 2, 3, 64)
    with pytest.raises(ValueError, match=r"v must be a torch.float32 CUDA tensor \[rows\]\[2\]\[64\]"):
        abg.kvq_put(k[:, :, :64], k[:, :, ::2], cache)
    with pytest.raises(ValueError, match="qo must be"):
        abg.kvq_put(k[:, :, :64], k[:, :, 64:], cache, q=k[:, :, :64], qo=torch.zeros(5, device="cuda"))
    with pytest.raises(abg.AbgError, match="misaligned"):
        abg.kvq_put(k[:, :, 1:65], k[:, :, 64:], cache)
    with pytest.raises(ValueError, match="a row for every slot"):
        abg.kvq_get(cache, k[:, :, :64], None, slots=i64([0, 1, 2, 0]))
    with pytest.raises(ValueError, match="k or v"):
        abg.kvq_get(cache, None, None)
    with pytest.raises(abg.AbgError, match="output overlaps"):
        abg.kvq_get(cache, k[:, :, :64], k[:, :, :64])
    with pytest.raises(abg.AbgError, match="output overlaps"):  # rows that lie in one another
        abg.kvq_get(cache, k[:, :1, :64].expand(3, 2, 64), None)
    abg.kvq_get(cache, k[:, :, :64], k[:, :, 64:])


# -------------------------------------------------------- the draft decoder ----
@pytest.mark.parametrize("cache", ["q4", "q8"])
@pytest.mark.parametrize("group", [32, 64])
def test_draft_decoder_over_a_quantised_cache(cache, group):
    """Trees whose one branch is the right continuation give the tokens of single
    steps; the cache holds what the steps' rows quantise to."""
    from affine_bit_group_gb300 import decode, draft, synth
    V, D = 1500, 64
    model, _ = synth.decode_model(seed=31, n_layers=2, hidden=512, mlp=1024, head_rows=V, q_rows=8 * D, kv_rows=2 * D)
    dm = decode.DeviceModel.upload(model)
    embed = dev(np.random.default_rng(32).standard_normal((V, 512)).astype(np.float32))

    def decoder():
        return draft.DraftDecoder(dm, embed, D=D, requests=2, pages=64, page=4, max_len=200, rows=40, cache=cache, group=group)

    one, tok, want = decoder(), i32([7, 1200]), []
    for _ in range(18):
        _, add, last = one.step(tok, i32([-1, -1]), i32([0, 1, 2]), 1)
        assert host(add).tolist() == [1, 1]
        tok = last.clone()
        want.append(host(tok))
    want = np.stack(want, 1)
    dec, first, at = decoder(), [7, 1200], 0
    for depth in (3, 1, 4, 2, 0):
        t, p = [], []
        for b in range(2):
            chain = [first[b] if at == 0 else want[b, at - 1]] + [want[b, at + i] for i in range(depth)]
            wrong = [(want[b, at] + 1) % V]
            t += chain + wrong
            p += [-1] + list(range(depth)) + [0]
        n = depth + 2
        rows, add, last = dec.step(i32(t), i32(p), i32([0, n, 2 * n]), n)
        assert host(add).tolist() == [depth + 1] * 2
        at += depth + 1
        assert host(last).tolist() == want[:, at - 1].tolist()
    assert host(dec.lens[0]).tolist() == [at, at]
    # the rows of both ways of decoding are the same tokens' (the products' batches differ in no bit)
    for i in range(2):
        got = []
        for d in (one, dec):
            table = host(d.table)
            slots = np.concatenate([table[b, np.arange(at) // 4].astype(np.int64) * 4 + np.arange(at) % 4 for b in range(2)])
            k, v = (torch.empty((2 * at, 2, D), device="cuda") for _ in range(2))
            abg.kvq_get(d.caches[i], k, v, slots=i64(slots))
            got.append((k, v))
        if i == 0:  # the first layer's rows depend on the tokens and positions alone
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert abg.device_status(clear=True) == 0


@pytest.mark.parametrize("cache", ["q4", "q8"])
def test_draft_decoder_holds_the_rows_that_the_drafts_saw(cache):
    """Value rows far from 0 against their spread, whose bias rounds by many scales:
    quantised again after being read back they would have other codes."""
    from affine_bit_group_gb300 import decode, draft, synth
    V, D, n = 700, 64, 5
    model, _ = synth.decode_model(seed=41, n_layers=2, hidden=512, mlp=512, head_rows=V, q_rows=4 * D, kv_rows=2 * D)
    dm = decode.DeviceModel.upload(model)
    rng = np.random.default_rng(42)
    for L in dm.layers:  # all rows of V's matrix are its first one, but for one bias
        for t in (L["v"].w, L["v"].scale, L["v"].bias):
            m = t.view(2 * D, -1)
            m[:] = m[0].clone()
        L["v"].bias.view(2 * D, -1)[:, 0] += dev((1e-4 * rng.standard_normal(2 * D)).astype(np.float32)).to(L["v"].bias.dtype)
    embed = dev(rng.standard_normal((V, 512)).astype(np.float32))

    def decoder():
        return draft.DraftDecoder(dm, embed, D=D, requests=1, pages=8, page=4, max_len=32, rows=8, cache=cache)

    one, chain = decoder(), [7]
    for _ in range(n):
        chain.append(int(one.step(i32(chain[-1:]), i32([-1]), i32([0, 1]), 1)[2]))
    dec = decoder()
    rows, add, last = dec.step(i32(chain[:n]), i32(range(-1, n - 1)), i32([0, n]), n)
    assert host(rows).tolist() == list(range(n)) and host(add).tolist() == [n] and host(last).tolist() == chain[n:]
    # the last layer's drafts are still there
    table, t = host(dec.table)[0], np.arange(n)
    for held, cached in zip(dec.drafts, dec.caches[-1]):
        want, got = (host(x.view(torch.int32)) for x in (held, cached))
        assert np.array_equal(got[table[t // 4], :, t % 4], want[0, :, :n].swapaxes(0, 1))
    if cache == "q8":  # (and are such rows; in 4 bits these happen to keep their codes)
        k, v = (torch.empty((n, 2, D), device="cuda") for _ in range(2))
        abg.kvq_get(dec.drafts, k, v)
        again = abg.kvq_put(k, v, abg.kvq_cache(1, 2, 8, D, 8, 64))
        assert not torch.equal(again.Vc[:, :, :n], dec.drafts.Vc[:, :, :n])
