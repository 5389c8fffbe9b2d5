"""The draft-verification calls on the GPU against their plain forms: whole
numbers equal, kv_put's float32 rows bit for bit the single-token attention's
(the oracle), tree_attn within bounds derived from its roundings."""
from __future__ import annotations

import numpy as np
import pytest

import draft_ref as ref
import oracle
from affine_bit_group_gb300 import synth
from helpers import assert_bits_equal, dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
abg = pytest.importorskip("affine_bit_group_gb300")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U32 = 2.0**-24
UNIT = {"f32": U32, "bf16": 2.0**-8, "f16": 2.0**-11}  # largest relative rounding error


def i32(v):
    return dev(np.ascontiguousarray(v, np.int32))


def i64(v):
    return dev(np.ascontiguousarray(v, np.int64))


def wide(t):
    """A tensor's values in 64 bits."""
    return t.double().cpu().numpy()


# -------------------------------------------------------------- page_plan ----
def run_page_plan(lens, add, cu, held, ends, ring, table, page, N):
    B = len(lens)
    d = dict(ring=i32(ring), table=i32(table), slots=i64(np.full(N, 7)), pos=i32(np.full(N, 7)),
             lens=i32(np.full(B, 7)), held=i32(np.full(B, 7)), ends=i64([7, 7]), info=i32([7, 7]))
    want = ref.page_plan(lens, add, cu, held, ends, ring, table, page, N)
    for _ in range(2):  # reads nothing that it writes
        abg.page_plan(i32(lens), i32(add), i32(cu), i32(held), i64(ends), d["ring"], d["table"], page, d["slots"],
                      d["pos"], d["lens"], d["held"], d["ends"], d["info"])
        for k, v in want.items():
            assert np.array_equal(host(d[k]).reshape(v.shape), v), k
    return want


def plan_case(rng, B, page, width, most_len, most_add, prompt=False):
    lens = rng.integers(0, most_len + 1, B).astype(np.int32)
    span = rng.integers(0, most_add + 1, B)
    add = np.array([rng.integers(-1, s + 1) for s in span], np.int32)
    cu = np.concatenate([[0], np.cumsum(span)]).astype(np.int32)
    held = np.minimum(-(-lens // page) + rng.integers(0, 2, B), width).astype(np.int32)
    pool = int(held.sum()) + int(rng.integers(1, 2 * B * (most_add // page + 1)))
    order = rng.permutation(pool)
    table = rng.integers(-9, 0, (B, width)).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    head = int(rng.integers(0, 5 * pool))
    ring = np.full(pool, -3, np.int32)
    ring[(head + np.arange(pool - at)) % pool] = order[at:]
    return lens, add, cu, held, np.array([head, head + pool - at]), ring, table, page, int(cu[-1]) + 3


@pytest.mark.parametrize("B,page,width,most_len,most_add", [
    (1, 16, 4, 0, 1), (1, 1, 9, 5, 4), (7, 16, 8, 100, 8), (48, 16, 64, 900, 8), (513, 100, 12, 700, 300),
    (1500, 7, 40, 120, 20), (8192, 16, 6, 60, 3)])
def test_page_plan(B, page, width, most_len, most_add):
    rng = np.random.default_rng([B, page, width])
    for _ in range(3):
        run_page_plan(*plan_case(rng, B, page, width, most_len, most_add))


def test_page_plan_refusals_on_the_device():
    """Too few pages, a table row too short, a bad length, more tokens than the
    span, a bad page count: each refused alone, its neighbours granted."""
    lens = np.array([10, 60, -5, 3, 16, 4, 7, 2**31 - 2], np.int32)
    add = np.array([4, 8, 1, 5, 1, -1, -2, 1], np.int32)
    cu = np.array([0, 4, 12, 13, 17, 18, 18, 20, 22], np.int32)
    held = np.array([1, 4, 1, 1, 1, 9, 1, 1], np.int32)
    table = np.arange(32).reshape(8, 4).astype(np.int32)
    ring = np.arange(50, 55, dtype=np.int32)
    got = run_page_plan(lens, add, cu, held, np.array([2, 6]), ring, table, 16, 24)
    assert got["info"].tolist() == [1, 5]
    assert got["lens"].tolist() == [14, 60, -5, 3, 17, 4, 0, 2**31 - 2]
    # one free page, two requests that need one: the first has it
    got = run_page_plan(np.array([16, 16, 5], np.int32), np.array([1, 1, 1], np.int32), np.array([0, 1, 2, 3]),
                        np.array([1, 1, 1], np.int32), np.array([3, 4]), ring, table[:3], 16, 3)
    assert got["info"].tolist() == [1, 1] and got["slots"].tolist()[1] == -1


# -------------------------------------------------------------- tree_plan ----
def parents(rng, spans, wild=False):
    out = []
    for t in spans:
        p = np.array([-1 if i == 0 else rng.integers(max(-1, i - 8), i) for i in range(t)], np.int64)
        if wild and t:
            p = np.where(rng.random(t) < 0.3, rng.integers(-4, t + 4, t), p)  # any order, cycles, padding
        out.append(p)
    return np.concatenate(out + [np.zeros(0, np.int64)]).astype(np.int32)


@pytest.mark.parametrize("spans,words", [
    ([1], 1), ([2, 0, 5], 1), ([64, 63, 1], 1), ([65, 128, 100], 2), ([190, 192], 3), ([256, 0, 255, 7], 4),
    ([300, 20], 4), ([70, 3], 1)])
@pytest.mark.parametrize("wild", [False, True])
def test_tree_plan(spans, words, wild):
    rng = np.random.default_rng([len(spans), words, wild])
    cu = np.concatenate([[0], np.cumsum(spans)])
    N = int(cu[-1]) + 5
    parent = np.concatenate([parents(rng, spans, wild), np.zeros(5, np.int32)])
    lens = rng.integers(0, 1000, len(spans)).astype(np.int32)
    mask, pos = i64(np.full((N, words), 3)), i32(np.full(N, 3))
    abg.tree_plan(i32(parent), i32(lens), i32(cu), mask, pos)
    m, p = ref.tree_plan(parent, lens, cu, words)
    assert np.array_equal(host(mask), m)
    assert np.array_equal(host(pos), p)


def test_tree_plan_chain_of_the_largest_span():
    parent, lens = np.arange(-1, 255), np.array([9])
    mask, pos = i64(np.zeros((256, 4))), i32(np.zeros(256))
    abg.tree_plan(i32(parent), i32(lens), i32([0, 256]), mask, pos)
    assert np.array_equal(host(pos), 9 + np.arange(256))
    assert np.array_equal(host(mask), ref.pack(np.tri(256, dtype=bool)))


# ----------------------------------------------------------------- kv_put ----
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 256), (4, 4, 64), (16, 4, 128), (6, 3, 64)])
def test_kv_put_f32_is_the_single_token_steps_bit_for_bit(Hq, Hkv, D):
    """One token at position pos into an abg_atq cache (one page of P tokens)."""
    c = synth.atq_case(np.random.default_rng([Hq, Hkv, D, 1]), Hq, Hkv, D, 40, 17)
    Kc, Vc = dev(c["Kc"]), dev(c["Vc"])
    _, _, eK, eV = oracle.atq(**c)
    cos, sin = np.zeros((20, D // 2), np.float32), np.zeros((20, D // 2), np.float32)
    cos[17], sin[17] = c["cos"], c["sin"]
    qo = torch.empty((1, Hq, D), device="cuda")
    abg.kv_put(dev(c["k"]).view(1, Hkv, D), dev(c["v"]).view(1, Hkv, D), Kc.unsqueeze(0), Vc.unsqueeze(0),
               slots=i64([17]), q=dev(c["q"]).view(1, Hq, D), qo=qo, qn_w=dev(c["qn_w"]), kn_w=dev(c["kn_w"]),
               cos=dev(cos), sin=dev(sin), pos=i32([17]))
    assert_bits_equal(host(Kc), eK.reshape(host(Kc).shape), "K cache")
    assert_bits_equal(host(Vc), eV.reshape(host(Vc).shape), "V cache")
    want = ref.kv_put(c["q"].reshape(1, Hq, D), c["qn_w"], cos, sin, np.array([17]), 1e-6)
    # three roundings of the norm's factor, two products, a rotation of two products and a sum
    assert np.all(np.abs(host(qo) - want) <= 8 * U32 * np.abs(want).max() * 2)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,Hq,Hkv,D,page,norm,rope", [
    (1, 4, 4, 64, 1, True, True), (37, 6, 3, 64, 7, True, True), (130, 16, 4, 128, 16, True, False),
    (5, 8, 2, 256, 100, False, True), (64, 3, 1, 128, 48, False, False)])
def test_kv_put(kind, N, Hq, Hkv, D, page, norm, rope):
    rng = np.random.default_rng([N, Hq, D, page])
    T = TYPES[kind]
    pages = -(-N // page) + 1
    qkv = (1.5 * rng.standard_normal((N, Hq + 2 * Hkv, D))).astype(np.float32)
    slots = rng.permutation(pages * page)[:N].astype(np.int64)
    drop = rng.random(N) < 0.2
    slots[drop] = rng.choice([-1, -2**40, pages * page, 2**40], drop.sum())
    Kc, Vc = (torch.full((pages, Hkv, page, D), 3.0, dtype=T, device="cuda") for _ in range(2))
    qo = torch.empty((N, Hq, D), dtype=T, device="cuda")
    w = [(1 + 0.1 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2)]
    ang = rng.uniform(0, 6.28, (2 * N, D // 2))
    cs = [np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)] if rope else [None, None]
    pos = rng.integers(0, 2 * N, N)
    d = dev(qkv)
    opt = lambda x: None if x is None else dev(x)  # noqa: E731
    abg.kv_put(d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], Kc, Vc, slots=i64(slots), q=d[:, :Hq], qo=qo, qn_w=opt(w[0]),
               kn_w=opt(w[1]), cos=opt(cs[0]), sin=opt(cs[1]), pos=i32(pos) if rope else None)
    q = ref.kv_put(qkv[:, :Hq], w[0], *cs, pos, 1e-6)
    k = ref.kv_put(qkv[:, Hq:Hq + Hkv], w[1], *cs, pos, 1e-6)
    wantK, wantV = (np.full((pages * page, Hkv, D), 3.0) for _ in range(2))
    kept = (slots >= 0) & (slots < pages * page)
    wantK[slots[kept]], wantV[slots[kept]] = k[kept], qkv[kept, Hq + Hkv:]
    for got, want, what in ((wide(qo), q, "q"),
                            (wide(Kc).transpose(0, 2, 1, 3).reshape(wantK.shape), wantK, "K"),
                            (wide(Vc).transpose(0, 2, 1, 3).reshape(wantV.shape), wantV, "V")):
        # the f32 steps as above, then one rounding to the type
        bound = 16 * U32 * np.abs(want).max() + 1.01 * UNIT[kind] * np.abs(want) + 2.0**-25
        assert np.all(np.abs(got - want) <= bound), what


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_kv_put_moves_draft_rows_as_they_are(kind):
    """Accepted rows out of draft buffers [Hkv][rows][D], by index and slot."""
    rng = np.random.default_rng(3)
    T, Hkv, D, R = TYPES[kind], 3, 128, 29
    Kd, Vd = (torch.from_numpy(rng.standard_normal((Hkv, R, D))).to(T).cuda() for _ in range(2))
    Kc, Vc = (torch.zeros((4, Hkv, 10, D), dtype=T, device="cuda") for _ in range(2))
    rows = np.array([0, 28, 5, -1, 29, 6, 2**31 - 1, 7], np.int32)
    slots = np.array([39, 0, 11, 12, 13, -1, 14, 25], np.int64)
    abg.kv_put(Kd.transpose(0, 1), Vd.transpose(0, 1), Kc, Vc, rows=i32(rows), slots=i64(slots))
    for got, src in ((Kc, Kd), (Vc, Vd)):
        want = torch.zeros_like(got)
        for r, s in zip(rows, slots):
            if 0 <= r < R and 0 <= s < 40:
                want[s // 10, :, s % 10] = src[:, r]
        assert torch.equal(got, want)


def test_kv_put_position_outside_the_rotation_table_is_nan():
    k = torch.ones((3, 1, 64), device="cuda")
    Kc, Vc = (torch.zeros((1, 1, 3, 64), device="cuda") for _ in range(2))
    cs = torch.ones((5, 32), device="cuda")
    abg.kv_put(k, k, Kc, Vc, cos=cs, sin=torch.zeros_like(cs), pos=i32([4, 5, -1]))
    assert torch.equal(Kc[0, 0, 0], k[0, 0]) and torch.isnan(Kc[0, 0, 1:]).all() and torch.equal(Vc[0, 0], k[:, 0])


# -------------------------------------------------------------- tree_attn ----
def attn_case(seed, kind, Hq, Hkv, D, page, lens, spans, words=None, gate=True, y32=False, tail=2, qscale=2.0):
    """Inputs (device) of one call: random pages, masks of random trees, NaN in
    every cache row past a request's length, in the unused pages and in the
    draft rows past the spans."""
    rng = np.random.default_rng([seed, D, page])
    T = TYPES[kind]
    B, lens, spans = len(lens), np.array(lens), np.array(spans)
    words = words or max(1, -(-int(max(spans)) // 64))
    cu = np.concatenate([[0], np.cumsum(spans)])
    N = int(cu[-1]) + tail
    counts = -(-lens // page)
    pages, width = int(counts.sum()) + 2, int(max(1, counts.max()))
    order = rng.permutation(pages)
    table = rng.choice([-1, pages, 2**31 - 1, -2**31], (B, width))
    Kc, Vc = (rng.standard_normal((pages, Hkv, page, D)) for _ in range(2))
    used = np.zeros((pages, page), bool)
    at = 0
    for b in range(B):
        table[b, :counts[b]] = order[at:at + counts[b]]
        at += counts[b]
        t = np.arange(lens[b])
        used[table[b, t // page], t % page] = True
    for x in (Kc, Vc):
        x.transpose(0, 2, 1, 3)[~used] = np.nan
    Kd, Vd = (rng.standard_normal((Hkv, N + 3, D)) for _ in range(2))
    Kd[:, cu[-1]:] = Vd[:, cu[-1]:] = np.nan
    parent = np.concatenate([parents(rng, spans), np.full(tail, -2, np.int32)])
    mask, _ = ref.tree_plan(parent, lens, cu, words)
    t = lambda x: torch.from_numpy(x).to(T).cuda()  # noqa: E731
    return dict(q=t(qscale * rng.standard_normal((N, Hq, D))), Kc=t(Kc), Vc=t(Vc), table=i32(table), lens=i32(lens),
                cu=i32(cu), Kd=t(Kd), Vd=t(Vd), mask=i64(mask), max_span=int(max(1, min(max(spans), 64 * words))),
                gate=dev(rng.standard_normal((N, Hq, D)).astype(np.float32)) if gate else None,
                y=torch.full((N, Hq, D), 5.0, dtype=torch.float32 if y32 else T, device="cuda")), kind


def bits_of(mask):
    return np.unpackbits(host(mask).view(np.uint8), axis=1, bitorder="little").astype(bool)


def check_attn(c, kind, ysum=False, calls=1):
    c = dict(c)
    if ysum:
        c["ysum"] = torch.full((c["y"].numel() // 64,), 5.0, device="cuda")
    for _ in range(calls):
        abg.tree_attn(**c)
    w = {k: None if c[k] is None else wide(c[k]) for k in ("q", "Kc", "Vc", "Kd", "Vd", "gate")}
    bits = bits_of(c["mask"])
    want, terms = ref.tree_attn(w["q"], w["Kc"], w["Vc"], host(c["table"]), host(c["lens"]), host(c["cu"]), w["Kd"],
                                w["Vd"], bits, w["gate"])
    got = wide(c["y"])
    cu, cap = host(c["cu"]), bits.shape[1]
    written = np.zeros(len(got), bool)
    for b in range(len(cu) - 1):
        written[cu[b]:min(cu[b + 1], cu[b] + cap)] = True
    assert np.all(got[~written] == 5.0)
    # f32 steps: a score's D+2 roundings (each of its sum of magnitudes; it
    # moves a weight by as much, numerator and denominator), the weight itself
    # and its place in the sum, the joins of at most 600 pieces, the gate
    D, n = w["q"].shape[2], int(host(c["lens"]).max()) + cap
    top, mag = terms[..., :1], terms[..., 1:]
    bound = U32 * top * (2 * (D + 4) * mag + 2 * (64 + n / 16 + 600))
    if kind != "f32":
        bound += UNIT[kind] * top * 1.01  # the weights' rounding
        if c["y"].dtype != torch.float32:
            bound = bound + UNIT[kind] * np.abs(want) * 1.02 + 2.0**-25  # y's own
    err = np.abs(got - want)
    ok = (err <= bound) | (np.isnan(got) & np.isnan(want)) | (got == want)
    assert ok[written].all(), (np.argwhere(~ok & written[:, None, None])[:5], np.nanmax(err))
    if ysum:
        y = got.reshape(len(got), -1, 64)
        s = host(c["ysum"]).reshape(y.shape[:2]).astype(np.float64)
        assert np.all(np.abs(s - y.sum(2))[written] <= 64 * U32 * np.abs(y).sum(2)[written] + 1e-30)
        assert np.all(s[~written] == 5.0)
    return got, want


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
    (8, 2, 128, 128, [4000], [64]),
    (2, 2, 64, 100, [20000], [2]),
    (16, 1, 128, 24, [0, 0, 700], [20, 33, 40]),
]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,spans", ATTN)
def test_tree_attn(kind, Hq, Hkv, D, page, lens, spans):
    check_attn(*attn_case(1, kind, Hq, Hkv, D, page, lens, spans, gate=D != 128))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,spans", [
    (5, 1, [1, 1, 1, 1, 0, 1]), (8, 1, [1, 1, 1, 1, 1, 1]), (4, 2, [4, 1, 3, 0, 2, 4]), (6, 2, [2, 2, 1, 2, 2, 1]),
    (9, 1, [1, 1, 1, 1, 1, 1]), (8, 2, [4, 3, 1, 2, 4, 4]), (3, 3, [16, 9, 8, 5, 4, 11]), (17, 1, [1, 1, 1, 1, 1, 1]),
])
def test_tree_attn_few_rows_and_tiles_that_end_inside(D, Hq, Hkv, spans):
    """5 to 17 rows a key/value head, lengths around the tiles' ends."""
    check_attn(*attn_case(21, "f32", Hq, Hkv, D, 16, [31, 33, 64, 127, 129, 300], spans))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("spans", [[65, 128], [150, 1, 192], [256, 30]])
def test_tree_attn_spans_past_one_mask_word(kind, spans):
    check_attn(*attn_case(2, kind, 8, 2, 128, 16, [200, 33, 150][:len(spans)], spans))
    check_attn(*attn_case(3, kind, 3, 1, 256, 16, [130, 1, 0][:len(spans)], spans, gate=False))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_tree_attn_f32_result_and_group_sums(kind):
    check_attn(*attn_case(4, kind, 8, 2, 256, 16, [700, 15], [8, 3], y32=True), ysum=True)
    check_attn(*attn_case(5, kind, 4, 2, 64, 16, [9000], [4], y32=True), ysum=True)
    check_attn(*attn_case(6, kind, 16, 4, 128, 16, [300, 100], [40, 20], y32=True, gate=False), ysum=True)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_tree_attn_many_ragged_requests(kind):
    rng = np.random.default_rng(8)
    lens, spans = rng.integers(0, 700, 300), rng.integers(0, 6, 300)
    check_attn(*attn_case(7, kind, 4, 2, 64, 16, lens, spans))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_tree_attn_rows_that_see_nothing_are_zero(kind):
    """Padding drafts of a request without cached tokens, and with some."""
    c, k = attn_case(9, kind, 4, 2, 128, 16, [0, 40, 0], [6, 5, 70], gate=False)
    mask = host(c["mask"]).copy()
    mask[[2, 3, 7, 12, 60]] = 0
    mask[20, 0] = 0  # its only bits lie in the second word, if any
    c["mask"] = i64(mask)
    got, _ = check_attn(c, k)
    assert np.all(got[[2, 3, 12, 60]] == 0) and np.all(np.abs(got[7]).max(1) > 0)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 256])
def test_tree_attn_what_a_draft_does_not_see_does_not_reach_it(kind, D):
    """NaN and infinities in K and V of one draft: only the drafts that see it
    may show them."""
    c, k = attn_case(10, kind, 6, 3, D, 16, [50, 0], [40, 90])
    bits = bits_of(c["mask"])
    Kd, Vd = c["Kd"].clone(), c["Vd"].clone()
    clean = dict(c, Kd=Kd, Vd=Vd)
    bad = {5: (float("nan"), 1.0), 17: (1.0, float("nan")), 30: (1.0, float("inf")), 47: (float("inf"), 1.0),
           110: (1.0, float("-inf"))}
    for n, (fk, fv) in bad.items():
        clean["Kd"][:, n, 3] *= fk
        clean["Vd"][:, n, 7] *= fv
    abg.tree_attn(**clean)
    got = wide(clean["y"]).copy()
    for b, (lo, hi) in enumerate(((0, 40), (40, 130))):
        sees = np.array([[n - lo < hi - lo and lo <= n < hi and bits[t, n - lo] for n in bad] for t in range(lo, hi)])
        plain = ~sees.any(1)
        assert np.isfinite(got[lo:hi][plain]).all()
        # a NaN key: the whole row
        nan_key = sees[:, 0]
        assert np.isnan(got[lo:hi][nan_key]).all()
        only_v = sees[:, 1] & ~sees[:, 0] & ~sees[:, 3]
        assert np.isnan(got[lo:hi][only_v][..., 7]).all()
        assert np.isfinite(got[lo:hi][only_v][..., 8]).all()
    check_attn(dict(c, Kd=torch.where(torch.isfinite(Kd), Kd, 0), Vd=torch.where(torch.isfinite(Vd), Vd, 0)), k)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_tree_attn_scores_far_apart(kind):
    """Scores that grow along the sequence (every tile raises the maximum) and
    that fall, over +-200."""
    for sign in (1.0, -1.0):
        c, k = attn_case(11, kind, 4, 2, 128, 16, [1500], [6], gate=False)
        ramp = torch.linspace(-1, 1, 1500, device="cuda") * sign
        t = np.arange(1500)
        table = host(c["table"])[0]
        K = c["Kc"].clone()
        K[table[t // 16], :, t % 16, 0] = (ramp * 14).to(K.dtype)[:, None]
        q = c["q"].clone()
        q[..., 0] = 160.0
        check_attn(dict(c, Kc=K, q=q), k)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_tree_attn_bad_pages_read_as_zeros(kind):
    c, k = attn_case(12, kind, 4, 2, 64, 16, [200, 100], [3, 3])
    table = host(c["table"]).copy()
    table[0, 2], table[1, 0], table[0, 5] = -7, 2**31 - 1, -2**31
    check_attn(dict(c, table=i32(table)), k)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_tree_attn_is_the_same_on_every_run_and_on_other_streams(kind):
    c, k = attn_case(13, kind, 8, 2, 128, 16, [5000, 70, 900], [20, 3, 9])
    abg.tree_attn(**c)
    first = c["y"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    ws = [torch.empty(abg.tree_attn_workspace(c["q"], c["Kc"], c["max_span"]), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    for i in range(20):
        y = torch.empty_like(first)
        s = side if i % 2 else torch.cuda.current_stream()
        abg.tree_attn(**dict(c, y=y), ws=ws[i % 2], stream=s)
        outs.append(y)
    torch.cuda.synchronize()
    written = int(host(c["cu"])[-1])
    for y in outs:
        assert torch.equal(y[:written], first[:written])


def test_tree_attn_of_one_draft_is_the_single_token_attention():
    """f32, one page of P tokens, one draft a request, gate and group sums: the
    single-token oracle's step within f32 rounding (its order of sums differs)."""
    c = synth.atq_case(np.random.default_rng(21), 8, 2, 128, 400, 300)
    ey, eys, eK, eV = oracle.atq(**c)
    qo = torch.empty((1, 8, 128), device="cuda")
    Kd, Vd = (torch.empty((2, 1, 128), device="cuda") for _ in range(2))
    abg.kv_put(dev(c["k"]).view(1, 2, 128), dev(c["v"]).view(1, 2, 128), Kd.unsqueeze(0), Vd.unsqueeze(0),
               q=dev(c["q"]).view(1, 8, 128), qo=qo, qn_w=dev(c["qn_w"]), kn_w=dev(c["kn_w"]),
               cos=dev(c["cos"]).view(1, 64), sin=dev(c["sin"]).view(1, 64), pos=i32([0]))
    y, ys = torch.empty((1, 8, 128), device="cuda"), torch.empty((1, 16), device="cuda")
    abg.tree_attn(qo, dev(c["Kc"]).unsqueeze(0), dev(c["Vc"]).unsqueeze(0), i32([[0]]), i32([300]), i32([0, 1]), Kd, Vd,
                  i64([[1]]), y, gate=dev(c["gate"]).view(1, 8, 128), ysum=ys)
    assert_bits_equal(host(Kd)[:, 0], eK.reshape(2, 400, 128)[:, 300], "the draft's key row")
    # both sides within the f32 bound of check_attn of the exact value
    tol = 2 * U32 * np.abs(c["Vc"]).max() * (2 * 132 * 20 + 2 * 700)
    assert np.abs(host(y).ravel() - ey).max() <= tol
    assert np.abs(host(ys).ravel() - eys).max() <= 64 * tol


# ------------------------------------------------------------ tree_accept ----
def accept_case(rng, spans, V, tail=2):
    cu = np.concatenate([[0], np.cumsum(spans)])
    N = int(cu[-1]) + tail
    x = rng.standard_normal((N, V)).astype(np.float32)
    parent = np.concatenate([parents(rng, spans), np.full(tail, -1, np.int32)])
    parent[cu[:-1][np.array(spans) > 0]] = -1
    tok = rng.integers(0, V, N).astype(np.int32)
    best = x.argmax(1)
    for b, t in enumerate(spans):
        for i in range(1, t):
            if parent[cu[b] + i] >= 0 and rng.random() < 0.7:
                tok[cu[b] + i] = best[cu[b] + parent[cu[b] + i]]
    return x, tok, parent, cu


def run_accept(x, tok, parent, cu, device_x=None):
    N, B = len(tok), len(cu) - 1
    best, rows, add, last = i32(np.full(N, 9)), i32(np.full(N, 9)), i32(np.full(B, 9)), i32(np.full(B, 9))
    abg.tree_accept(dev(x) if device_x is None else device_x, i32(tok), i32(parent), i32(cu), best, rows, add, last)
    for got, want, what in zip((best, rows, add, last), ref.tree_accept(x, tok, parent, cu),
                               ("best", "rows", "add", "last")):
        assert np.array_equal(host(got), want), what


@pytest.mark.parametrize("spans,V", [([1], 1), ([3], 2), ([8], 31999), ([24, 0, 5, 60], 1003), ([256, 7], 4097),
                                     ([300, 1], 64), ([2] * 50, 12289)])
def test_tree_accept(spans, V):
    run_accept(*accept_case(np.random.default_rng([len(spans), V]), spans, V))


def test_tree_accept_ties_infinities_nan_and_strides():
    rng = np.random.default_rng(2)
    x, tok, parent, cu = accept_case(rng, [9, 6], 5003)
    x[0] = 1.5                                   # all equal: the lowest index
    x[1, [17, 4000]] = 88.0                      # a tie
    x[2, [6, 4999]] = np.inf
    x[3, :] = -np.inf                            # index 0
    x[4, :] = np.nan
    x[5, ::2] = np.nan
    x[6, :] = 0.0
    x[6, 3:] = -0.0                              # -0 is 0
    x[7, :], x[7, 4321] = -np.inf, -3e38
    x[8, :] = np.nan
    x[8, 77] = -np.inf                           # a NaN is -infinity: index 0
    run_accept(x, tok, parent, cu)
    big = torch.zeros((len(x), 5011), device="cuda")
    big[:, 3:5006] = dev(x)
    run_accept(x, tok, parent, cu, device_x=big[:, 3:5006])  # odd row stride, 12 bytes off a quad


def test_tree_accept_takes_the_first_right_child():
    x = np.zeros((6, 8), np.float32)
    x[[0, 1, 2, 3, 4, 5], [3, 4, 5, 6, 7, 1]] = 1
    run_accept(x, np.array([0, 2, 3, 3, 5, 6]), np.array([-1, 0, 0, 0, 2, 3]), np.array([0, 6]))
    # a parent that comes after its child, is itself, or is out of range is none
    run_accept(x, np.array([0, 3, 3, 3, 3, 3]), np.array([-1, 3, 2, 9, -7, 5]), np.array([0, 6]))


# ---------------------------------------------------------------- capture ----
def test_calls_record_into_a_cuda_graph():
    c, kind = attn_case(30, "bf16", 8, 2, 128, 16, [300, 90], [6, 4], tail=0)
    x, tok, parent, cu = accept_case(np.random.default_rng(4), [6, 4], 3001, tail=0)
    N, B = 10, 2
    xd, td, pd, cud = dev(x), i32(tok), i32(parent), i32(cu)
    mask, pos = i64(np.zeros((N, 1))), i32(np.zeros(N))
    best, rows, add, last = i32(np.zeros(N)), i32(np.zeros(N)), i32(np.zeros(B)), i32(np.zeros(B))
    ws = torch.empty(abg.tree_attn_workspace(c["q"], c["Kc"], c["max_span"]), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(abg.tree_accept_workspace(xd), dtype=torch.uint8, device="cuda")

    def step():
        abg.tree_plan(pd, c["lens"], cud, mask, pos)
        abg.tree_attn(**dict(c, mask=mask), ws=ws)
        abg.tree_accept(xd, td, pd, cud, best, rows, add, last, ws=ws2)

    step()
    want = c["y"].clone(), rows.clone(), add.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c["y"].fill_(5.0), rows.zero_(), add.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c["y"], want[0]) and torch.equal(rows, want[1]) and torch.equal(add, want[2])


# ---------------------------------------------------------------- refusals ----
def test_binding_refuses_wrong_tensors_on_the_device():
    c, _ = attn_case(40, "bf16", 4, 2, 64, 16, [20], [3], tail=0)
    ws = torch.empty(abg.tree_attn_workspace(c["q"], c["Kc"], c["max_span"]), dtype=torch.uint8, device="cuda")
    for change, words in ((dict(q=c["q"].float()), "q must be a contiguous torch.bfloat16"),
                          (dict(q=c["q"].transpose(0, 1)), "q must be"), (dict(q=c["q"][:, :, :32]), "q must be"),
                          (dict(lens=c["lens"].long()), "lens must be a contiguous torch.int32"),
                          (dict(mask=c["mask"][:, 0]), "mask must be"), (dict(mask=c["mask"][:2]), "mask must be"),
                          (dict(gate=c["gate"][:2]), "gate must be a contiguous torch.float32 CUDA tensor of at least"),
                          (dict(Kd=c["Kd"][:, :, :32]), "q must be"), (dict(y=c["y"].int()), "y must be float32"),
                          (dict(ws=ws.int()), "ws must be a contiguous torch.uint8"), (dict(cu=c["cu"][:1]), "cu must be")):
        with pytest.raises(ValueError, match=words):
            abg.tree_attn(**{**c, "ws": ws, **change})
    with pytest.raises(abg.AbgError, match="bad shape"):
        abg.tree_attn(**dict(c, ws=ws[:64]))
    with pytest.raises(abg.AbgError, match="output overlaps"):
        abg.tree_attn(**dict(c, y=c["q"], ws=ws))
    k = torch.zeros((3, 2, 128), device="cuda")
    Kc, Vc = (torch.zeros((1, 2, 3, 64), device="cuda") for _ in range(2))
    with pytest.raises(ValueError, match=r"k must be a torch.float32 CUDA tensor \[rows\]\[2\]\[64\]"):
        abg.kv_put(k[:, :, ::2], k[:, :, ::2], Kc, Vc)
    with pytest.raises(ValueError, match="qo must be"):
        abg.kv_put(k[:, :, :64], k[:, :, 64:], Kc, Vc, q=k[:, :, :64], qo=torch.zeros(5, device="cuda"))
    with pytest.raises(abg.AbgError, match="misaligned"):
        abg.kv_put(k[:, :, 1:65], k[:, :, 64:], Kc, Vc)
    abg.kv_put(k[:, :, :64], k[:, :, 64:], Kc, Vc)  # rows and heads with strides of their own


# ------------------------------------------------------------- far offsets ----
@pytest.mark.parametrize("kind,pages", [("bf16", 70000), ("f32", 70000)])
def test_pages_past_two_to_the_31_elements(kind, pages):
    """A cache of more than 2^31 elements, its last pages in use: rows put there
    are found there."""
    T, Hkv, page, D = TYPES[kind], 4, 64, 128
    assert pages * Hkv * page * D > 2**31
    Kc, Vc = (torch.empty((pages, Hkv, page, D), dtype=T, device="cuda") for _ in range(2))
    n = 100
    table = np.array([[pages - 1, pages - 2]])
    k, v = (torch.randn((n, Hkv, D), device="cuda") for _ in range(2))
    t = np.arange(n)
    slots = table[0, t // page].astype(np.int64) * page + t % page
    abg.kv_put(k, v, Kc, Vc, slots=i64(slots))
    assert torch.equal(Kc[-1].transpose(0, 1), k[:page].to(T)) and torch.equal(Vc[-2, :, :n - page].transpose(0, 1), v[page:].to(T))
    c, _ = attn_case(50, kind, 8, 4, D, page, [n], [5], gate=False)
    c.update(Kc=Kc, Vc=Vc, table=i32(table))
    abg.tree_attn(**c)
    far = c["y"].clone()
    c.update(Kc=Kc[-2:].clone(), Vc=Vc[-2:].clone(), table=i32([[1, 0]]))
    abg.tree_attn(**c)
    assert torch.equal(far[:5], c["y"][:5])
    check_attn(c, kind)


def test_early_start_off_gives_the_same_bits(tmp_path):
    """ABG_PDL=0 in a process of its own: plain stream order, the same results."""
    import os
    import subprocess
    import sys
    prog = tmp_path / "run.py"
    prog.write_text(
        "import sys, torch\n"
        f"sys.path[:0] = {[os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__))]!r}\n"
        "import test_gpu_9_draft as t\n"
        "out = []\n"
        "for kind in ('f32', 'bf16'):\n"
        "    c, _ = t.attn_case(60, kind, 8, 2, 128, 16, [900, 40], [9, 30], tail=0)\n"
        "    t.abg.tree_attn(**c)\n"
        "    out.append(c['y'].cpu())\n"
        "x, tok, parent, cu = t.accept_case(t.np.random.default_rng(1), [9, 30], 5000, tail=0)\n"
        "r = [t.i32(t.np.zeros(39)), t.i32(t.np.zeros(39)), t.i32([0, 0]), t.i32([0, 0])]\n"
        "t.abg.tree_accept(t.dev(x), t.i32(tok), t.i32(parent), t.i32(cu), *r)\n"
        "torch.save(out + [v.cpu() for v in r], sys.argv[1])\n")
    got = []
    for v in ("0", "1"):
        path = tmp_path / v
        env = dict(os.environ, ABG_PDL=v)
        subprocess.run([sys.executable, str(prog), str(path)], check=True, env=env, timeout=120)
        got.append(torch.load(path))
    assert all(torch.equal(a, b) for a, b in zip(*got))
