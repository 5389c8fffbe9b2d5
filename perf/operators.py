"""Cases that time the draft-verification operators, with their plain forms.

A decoder that checks several guessed tokens per step runs, for each step,
`page_plan` (pages and cache slots for the tokens that were accepted),
`tree_plan` (ancestor masks and positions of the new draft trees), `kv_put`
(norm, rotation and cache layout of q, k and v), `tree_attn` (attention of the
drafts over the paged cache and their own ancestors) and `tree_accept` (the
longest path of drafts that the logits agree with).  Head counts and widths are
those of this repository's mixer tests and synthetic decode token (8 heads over
2 of 256 columns, 16 over 2, 16 over 4, 6 over 3, 8 over 1), its 248320-row
head, and the eight tokens its batched product takes at a time; the rest is
generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HEADS = ((8, 2), (16, 2), (16, 4), (6, 3), (8, 1), (4, 4))
EPS = 1e-6


def listed():
    return [
        # one sequence, one token, the f32 cache of the single-token mixer: latency
        dict(name="attn one token f32", op="attn", type="f32", B=1, T=1, Hq=8, Hkv=2, D=256, L=2047, ragged=0.0,
             page=64, gate=True),
        # four sequences of eight drafts (one batched product), f32 throughout
        dict(name="attn drafts f32", op="attn", type="f32", B=4, T=8, Hq=16, Hkv=2, D=256, L=4100, ragged=0.5,
             page=32, gate=True),
        # a serving batch of trees over long, ragged sequences in small pages
        dict(name="attn trees bf16", op="attn", type="bf16", B=32, T=24, Hq=16, Hkv=4, D=128, L=12000, ragged=0.5,
             page=16, gate=False),
        # one very long sequence with a wide tree
        dict(name="attn long tree f16", op="attn", type="f16", B=1, T=63, Hq=16, Hkv=2, D=128, L=131071, ragged=0.0,
             page=128, gate=False),
        # a decode step's accepted tokens: few tokens, latency
        dict(name="pages step", op="pages", B=48, T=8, L=4096, page=16, width=512, prompt=False),
        # a wave of prompts admitted at once
        dict(name="pages prompts", op="pages", B=512, T=1500, L=0, page=16, width=128, prompt=True),
        # one tree, and a batch of trees past one mask word
        dict(name="trees one", op="trees", B=1, T=60, words=1, ragged=0.0),
        dict(name="trees batch", op="trees", B=256, T=120, words=2, ragged=0.5),
        # the drafts of a step: norm, rotation, into rows of their own
        dict(name="put drafts", op="put", type="f32", N=32, Hq=8, Hkv=2, D=256, page=0, norm=True, copy=False),
        # a long prompt into 16-bit pages
        dict(name="put prompt", op="put", type="bf16", N=8191, Hq=16, Hkv=4, D=128, page=16, norm=True, copy=False),
        # the greedy check of one sequence's drafts, and of a batch's, over the full head
        dict(name="accept one", op="accept", B=1, T=8, V=248320, ragged=0.0),
        dict(name="accept batch", op="accept", B=16, T=24, V=248320, ragged=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "pages", "trees", "put", "accept"])
    if op == "attn":
        kind = rng.choice(["f32", "bf16", "f16"])
        Hq, Hkv = rng.choice(HEADS)
        D = rng.choice([64, 128, 256])
        c = dict(op=op, type=kind, B=_log(rng, 1, 64), T=_log(rng, 1, 16 if kind == "f32" else 64), Hq=Hq, Hkv=Hkv,
                 D=D, L=_log(rng, 16, 131071), ragged=rng.choice([0.0, 0.5, 0.9]), page=rng.choice([16, 32, 64, 100, 128]),
                 gate=rng.random() < 0.5)
        while True:  # no more than the largest listed ones read and compute
            w = work(c)
            if w["bytes"] <= 4e8 and w["flops"] <= (2e10 if kind == "f32" else 6e10) and \
                    c["B"] * Hq * c["T"] * c["L"] <= 1.3e8:
                return c
            if c["L"] > 512:
                c["L"] = c["L"] * 2 // 3
            else:
                c["B"] = max(1, c["B"] // 2)
    if op == "pages":
        prompt = rng.random() < 0.5
        return dict(op=op, B=_log(rng, 1, 600), T=_log(rng, 16, 1500) if prompt else rng.randint(1, 16),
                    L=0 if prompt else _log(rng, 16, 8000), page=rng.choice([16, 32, 64, 100]), width=512,
                    prompt=prompt)
    if op == "trees":
        T = _log(rng, 1, 250)
        return dict(op=op, B=_log(rng, 1, 120), T=T, words=(T + 63) // 64, ragged=rng.choice([0.0, 0.5]))
    if op == "put":
        Hq, Hkv = rng.choice(HEADS)
        copy = rng.random() < 0.25
        return dict(op=op, type=rng.choice(["f32", "bf16", "f16"]), N=_log(rng, 1, 4000), Hq=Hq, Hkv=Hkv,
                    D=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 100]) if copy else rng.choice([0, 16, 32, 100]),
                    norm=not copy and rng.random() < 0.8, copy=copy)
    return dict(op=op, B=_log(rng, 1, 16), T=_log(rng, 1, 24), V=_log(rng, 31999, 248320), ragged=rng.choice([0.0, 0.5]))


# ----------------------------------------------------------------- sizes ----
def _lens(c):
    """Cached tokens of each sequence (a fixed ragged pattern of the case)."""
    return [int(round(c["L"] * (1.0 - c["ragged"] * ((b + 1) * 0.6180339887 % 1.0)))) for b in range(c["B"])]


def _spans(c):
    """Drafted tokens of each sequence."""
    if not c.get("ragged"):
        return [c["T"]] * c["B"]
    return [max(1, int(round(c["T"] * (1.0 - c["ragged"] * ((b + 1) * 0.7548776662 % 1.0))))) for b in range(c["B"])]


def _cu(spans):
    return np.concatenate([[0], np.cumsum(spans)])


def work(c):
    if c["op"] == "attn":
        e, D, Hq, Hkv = (4 if c["type"] == "f32" else 2), c["D"], c["Hq"], c["Hkv"]
        lens, spans = _lens(c), _spans(c)
        N = sum(spans)
        kv = 2 * Hkv * D * e * (sum(lens) + N)
        io = N * Hq * D * (2 * e + (4 if c["gate"] else 0)) + 8 * N
        return {"bytes": kv + io, "flops": 4 * D * Hq * sum(t * (n + (t + 1) / 2) for t, n in zip(spans, lens))}
    if c["op"] == "pages":
        N = c["B"] * c["T"]
        return {"bytes": 12 * N + c["B"] * 24, "flops": 0}
    if c["op"] == "trees":
        N = sum(_spans(c))
        return {"bytes": N * (4 + 8 * c["words"] + 4), "flops": 0}
    if c["op"] == "put":
        e = 4 if c["type"] == "f32" else 2
        src = e if c["copy"] else 4
        heads = 2 * c["Hkv"] + (0 if c["copy"] else c["Hq"])
        return {"bytes": c["N"] * (heads * c["D"] * (src + e) + 12 + (0 if c["copy"] else 4 * c["D"])), "flops": 0}
    N = sum(_spans(c))
    return {"bytes": 4 * N * (c["V"] + 4), "flops": 0}


# ---------------------------------------------------------------- inputs ----
def _i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


def _parents(rng, spans):
    """Local parent index of each draft: node 0 is the root, later ones hang off
    one of the eight before them."""
    return np.concatenate([[-1 if i == 0 else int(rng.integers(max(0, i - 8), i)) for i in range(t)] for t in spans])


def _ancestors(parent, spans, words):
    """Mask words [N][words]: bit j of a node says that it is j or below j."""
    out = np.zeros((len(parent), words), np.uint64)
    at = 0
    for t in spans:
        for i in range(t):
            p = parent[at + i]
            if p >= 0:
                out[at + i] = out[at + p]
            out[at + i, i // 64] |= np.uint64(1 << (i % 64))
        at += t
    return torch.from_numpy(out.view(np.int64)).cuda()


def prepare(c, seed):
    rng = np.random.default_rng([seed, 17])
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        t = torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)
        return t

    s = dict(case=c, op=c["op"])
    if c["op"] == "attn":
        T = TYPES[c["type"]]
        B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
        lens, spans = _lens(c), _spans(c)
        N = sum(spans)
        counts = [-(-n // page) for n in lens]
        pages, width = sum(counts) + 3, max(1, max(counts))
        order = rng.permutation(pages)
        table = np.full((B, width), -1)
        at = 0
        for b, n in enumerate(counts):
            table[b, :n] = order[at:at + n]
            at += n
        words = (max(spans) + 63) // 64
        s.update(q=normal(N, Hq, D, scale=2.0, dtype=T), Kc=normal(pages, Hkv, page, D, dtype=T),
                 Vc=normal(pages, Hkv, page, D, dtype=T), Kd=normal(Hkv, N, D, dtype=T), Vd=normal(Hkv, N, D, dtype=T),
                 gate=normal(N, Hq, D) if c["gate"] else None, table=_i32(table), lens=_i32(lens),
                 cu=_i32(_cu(spans)), mask=_ancestors(_parents(rng, spans), spans, words),
                 max_len=max(lens), max_span=max(spans), y=torch.empty((N, Hq, D), dtype=T, device="cuda"),
                 ysum=torch.empty((N, Hq * D // 64), device="cuda") if T == torch.float32 else None)
    elif c["op"] == "pages":
        B, T, page, width = c["B"], c["T"], c["page"], c["width"]
        lens = np.zeros(B, np.int64) if c["prompt"] else rng.integers(c["L"] // 2, c["L"] + 1, B)
        add = np.full(B, T) - rng.integers(0, T // 2 + 1, B) if c["prompt"] else rng.integers(0, T + 1, B)
        add[B // 2::7] = -1 if not c["prompt"] else add[B // 2::7]  # some sequences have ended
        held = -(-lens // page)
        pool = B * -(-(c["L"] + T) // page) + 5  # enough for every sequence at its longest
        order = rng.permutation(pool)
        table = np.full((B, width), -1)
        at = 0
        for b in range(B):
            table[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
        head = int(rng.integers(0, 10 * pool))
        ring = np.full(pool, -1)
        ring[(head + np.arange(pool - at)) % pool] = order[at:]
        N = B * T
        s.update(lens=_i32(lens), add=_i32(add), cu=_i32(T * np.arange(B + 1)), held=_i32(held),
                 ends=torch.tensor([head, head + pool - at], dtype=torch.int64, device="cuda"), ring=_i32(ring),
                 table=_i32(table), page=page, slots=torch.empty(N, dtype=torch.int64, device="cuda"),
                 pos=_i32(np.zeros(N)), lens_out=_i32(lens), held_out=_i32(held), info=_i32([0, 0]),
                 ends_out=torch.zeros(2, dtype=torch.int64, device="cuda"))
    elif c["op"] == "trees":
        spans = _spans(c)
        N = sum(spans)
        s.update(parent=_i32(_parents(rng, spans)), lens=_i32(rng.integers(0, 10000, c["B"])), cu=_i32(_cu(spans)),
                 max_span=max(spans), words=c["words"],
                 mask=torch.empty((N, c["words"]), dtype=torch.int64, device="cuda"), pos=_i32(np.zeros(N)))
    elif c["op"] == "put":
        T = TYPES[c["type"]]
        N, Hq, Hkv, D, page = c["N"], c["Hq"], c["Hkv"], c["D"], c["page"]
        if page:
            pages = -(-N // page) + 2
            start = int(rng.integers(0, page))
            order = rng.permutation(pages)
            p = start + np.arange(N)
            slots = order[p // page] * page + p % page
            slots[rng.random(N) < 0.02] = -1  # tokens that are not kept
            if c["copy"]:
                slots[rng.random(N) < 0.5] = -1
            s["slots"] = torch.as_tensor(slots, dtype=torch.int64).cuda()
        else:
            pages, page, s["slots"] = 1, N, None
        s.update(Kc=torch.zeros((pages, Hkv, page, D), dtype=T, device="cuda"),
                 Vc=torch.zeros((pages, Hkv, page, D), dtype=T, device="cuda"))
        if c["copy"]:  # accepted drafts into the cache: rows of the draft buffers, as they are
            rows = np.sort(rng.permutation(2 * N)[:N])
            s.update(k=normal(Hkv, 2 * N, D, dtype=T).transpose(0, 1), v=normal(Hkv, 2 * N, D, dtype=T).transpose(0, 1),
                     rows=_i32(rows))
        else:
            qkv = normal(N, Hq + 2 * Hkv, D, scale=1.5)  # one product's output
            ang = torch.rand((N + 999, D // 2), device="cuda", generator=gen) * (2 * math.pi)
            s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], cos=ang.cos(), sin=ang.sin(),
                     pos=_i32(int(rng.integers(0, 1000)) + np.arange(N)),
                     qo=torch.empty((N, Hq, D), dtype=T, device="cuda"))
            if c["norm"]:
                s.update(qn_w=1 + normal(D, scale=0.1), kn_w=1 + normal(D, scale=0.1))
    else:
        spans, V = _spans(c), c["V"]
        N = sum(spans)
        parent, cu = _parents(rng, spans), _cu(spans)
        want = rng.integers(0, V, N)
        tok = rng.integers(0, V, N)
        first = np.repeat(cu[:-1], spans)
        for n in np.nonzero(parent >= 0)[0]:  # most drafts guess right
            if rng.random() < 0.7:
                tok[n] = want[first[n] + parent[n]]
        logits = normal(N, V)
        logits[torch.arange(N, device="cuda"), torch.as_tensor(want).cuda()] = 9.0
        s.update(logits=logits, tok=_i32(tok), parent=_i32(parent), cu=_i32(cu), max_span=max(spans),
                 best=_i32(np.zeros(N)), rows=_i32(np.zeros(N)), add=_i32(np.zeros(c["B"])),
                 last=_i32(np.zeros(c["B"])))
    return s


# ------------------------------------------------------------ plain forms ----
def _padded(s):
    """Row of draft t of request b [B][T], and whether there is one."""
    cu = s["cu"].long()
    t = torch.arange(s["max_span"], device="cuda")
    there = t < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + t, 0), there


def _plain_attn(s):
    Hkv, page, D = s["Kc"].shape[1:]
    N, Hq = s["q"].shape[:2]
    B, L, G = len(s["lens"]), s["max_len"], Hq // Hkv
    idx, there = _padded(s)
    T = idx.shape[1]
    at = torch.arange(L, device="cuda")
    pages = s["table"].long().clamp(min=0)[:, at // page]
    K = s["Kc"][pages, :, (at % page)[None]].permute(0, 2, 1, 3).float()
    V = s["Vc"][pages, :, (at % page)[None]].permute(0, 2, 1, 3).float()
    Kd, Vd = (s[n][:, idx].transpose(0, 1).float() for n in ("Kd", "Vd"))
    q = s["q"][idx].float().view(B, T, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, T * G, D)
    sees = (s["mask"][idx][:, :, torch.arange(T, device="cuda") // 64] >> (torch.arange(T, device="cuda") % 64)) & 1
    sees = (sees > 0) & there[:, None, :]
    sees = sees[:, None, :, None, :].expand(B, 1, T, G, T).reshape(B, 1, T * G, T)
    S = torch.cat([(q @ K.transpose(2, 3)).masked_fill_((at >= s["lens"][:, None])[:, None, None], -math.inf),
                   (q @ Kd.transpose(2, 3)).masked_fill_(~sees, -math.inf)], 3).mul_(D ** -0.5)
    m = S.amax(3, keepdim=True)
    p = S.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(3, keepdim=True)
    o = p[..., :L] @ V + p[..., L:] @ Vd
    o = torch.where(l > 0, o / l, 0.0).view(B, Hkv, T, G, D).transpose(1, 2).reshape(B, T, Hq, D)
    y = torch.zeros((N, Hq, D), device="cuda")
    y[idx[there]] = o[there]
    if s["gate"] is not None:
        y = y * (1.0 / (1.0 + torch.exp(-s["gate"])))
    if s["ysum"] is not None:
        return y, y.view(N, Hq * D // 64, 64).sum(2)
    return y.to(s["q"].dtype)


def _plain_pages(s):
    lens, add, held, table, page = s["lens"].long(), s["add"].long(), s["held"].long(), s["table"], s["page"]
    cu, ring, (B, width), R = s["cu"].long(), s["ring"], s["table"].shape, len(s["ring"])
    head, tail = s["ends"][0], s["ends"][1]
    gone = add < 0
    need = (lens + add + page - 1) // page
    bad = (lens < 0) | (held < 0) | (held > width) | (~gone & ((add > cu[1:] - cu[:-1]) | (need > width)))
    extra = torch.where(gone | bad, 0, (need - held).clamp(min=0))
    upto = extra.cumsum(0)
    ok = ~gone & ~bad & ((extra == 0) | (upto <= tail - head))
    base = upto - extra
    extra = torch.where(ok, extra, 0)
    freed = torch.where(gone & ~bad, held, 0)
    j = torch.arange(width, device="cuda")[None]
    fresh = (j >= held[:, None]) & (j < (held + extra)[:, None])
    new = torch.where(fresh, ring[((head + base - held)[:, None] + j) % R], table)
    to = torch.where(j < freed[:, None], (tail + (freed.cumsum(0) - freed)[:, None] + j) % R, R)
    ring = torch.cat([ring, ring[:1]]).scatter(0, to.flatten(), table.flatten())[:R]
    n = torch.arange(len(s["slots"]), device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), n, right=True).clamp(max=B - 1)
    i = n - cu[b]
    live = (n < cu[B]) & ok[b] & (i < add[b])
    p = torch.where(live, lens[b] + i, 0)
    slots = torch.where(live, new[b, p // page].long() * page + p % page, -1)
    done = gone & ~bad
    return dict(slots=slots, pos=p.int(), table=new, ring=ring,
                lens=torch.where(ok, lens + add, torch.where(done, 0, lens)).int(),
                held=torch.where(done, 0, held + extra).int(),
                ends=torch.stack([head + extra.sum(), tail + freed.sum()]),
                info=torch.stack([extra.sum(), (~ok & ~done).sum()]).int())


def _plain_trees(s):
    idx, there = _padded(s)
    T, W = idx.shape[1], s["words"]
    j = torch.arange(T, device="cuda")
    sees = ((s["parent"][idx][:, :, None] == j) | (j[:, None] == j)) & there[:, :, None]
    for _ in range(max(1, (T - 1).bit_length())):  # twice the distance to the root each time
        sees = sees.float() @ sees.float() > 0
    bits = torch.zeros((len(idx), T, 64 * W), dtype=torch.int64, device="cuda")
    bits[:, :, :T] = sees.long() << (j % 64)
    mask = torch.zeros((len(s["pos"]), W), dtype=torch.int64, device="cuda")
    mask[idx[there]] = bits.view(len(idx), T, W, 64).sum(3)[there]
    pos = torch.zeros_like(s["pos"])
    pos[idx[there]] = (s["lens"][:, None] + sees.sum(2) - 1).int()[there]
    return mask, pos


def _plain_rope(s, x, w):
    D = x.shape[2]
    if w is not None:
        x = x / (x.square().mean(2, keepdim=True) + EPS).sqrt() * w
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], 2)


def _plain_put(s):
    k, v, Kc, Vc = s["k"], s["v"], s["Kc"].clone(), s["Vc"].clone()
    N, page = s["case"]["N"], Kc.shape[2]
    if s["case"]["copy"]:
        k, v = k[s["rows"].long()], v[s["rows"].long()]
    else:
        k = _plain_rope(s, k, s.get("kn_w"))
    slots = torch.arange(N, device="cuda") if s["slots"] is None else s["slots"]
    kept = slots >= 0
    at = slots[kept]
    Kc[at // page, :, at % page] = k[kept].to(Kc.dtype)
    Vc[at // page, :, at % page] = v[kept].to(Kc.dtype)
    if s["case"]["copy"]:
        return Kc, Vc
    return Kc, Vc, _plain_rope(s, s["q"], s.get("qn_w")).to(Kc.dtype)


def _plain_accept(s):
    x = s["logits"]
    V = x.shape[1]
    best = torch.where(x == x.amax(1, keepdim=True), torch.arange(V, device="cuda"), V).amin(1)
    idx, there = _padded(s)
    B, T = idx.shape
    j = torch.arange(T, device="cuda")
    parent = torch.where(there, s["parent"][idx], -2).long()
    guess = s["tok"][idx] == best[idx].gather(1, parent.clamp(min=0))
    right = (parent[:, :, None] == j) & guess[:, :, None]  # [child][parent]
    right = right & (right.long().cumsum(1) == 1)  # the first right child of each
    reach = right | (j[:, None] == j)
    for _ in range(max(1, (T - 1).bit_length())):
        reach = reach.float() @ reach.float() > 0
    kept = reach[:, :, 0] & there
    add = kept.sum(1)
    order = torch.where(kept, j, T).sort(1).values
    rows = torch.full((len(s["rows"]),), -1, dtype=torch.int32, device="cuda")
    rows[idx[there]] = torch.where(order < T, s["cu"][:-1, None] + order, -1).int()[there]
    end = (order * (j == add[:, None] - 1)).sum(1)
    last = best[s["cu"][:-1].long() + end]
    return dict(best=best.int(), rows=rows, add=add.int(), last=last.int())


def _plain(s):
    return {"attn": _plain_attn, "pages": _plain_pages, "trees": _plain_trees, "put": _plain_put,
            "accept": _plain_accept}[s["op"]](s)


# -------------------------------------------------------------- the calls ----
def run(s):
    if not own:
        return _plain(s)
    import affine_bit_group_gb300 as abg
    op = s["op"]
    if op == "attn":
        if "ws" not in s:  # kept with the buffers, as a decoding loop does
            s["ws"] = torch.empty(abg.tree_attn_workspace(s["q"], s["Kc"], s["max_span"]), dtype=torch.uint8,
                                  device="cuda")
        abg.tree_attn(s["q"], s["Kc"], s["Vc"], s["table"], s["lens"], s["cu"], s["Kd"], s["Vd"], s["mask"], s["y"],
                      max_span=s["max_span"], gate=s["gate"], ysum=s["ysum"], ws=s["ws"])
        return s["y"] if s["ysum"] is None else (s["y"], s["ysum"])
    if op == "pages":
        abg.page_plan(s["lens"], s["add"], s["cu"], s["held"], s["ends"], s["ring"], s["table"], s["page"], s["slots"],
                      s["pos"], s["lens_out"], s["held_out"], s["ends_out"], s["info"])
        return dict(slots=s["slots"], pos=s["pos"], table=s["table"], ring=s["ring"], lens=s["lens_out"],
                    held=s["held_out"], ends=s["ends_out"], info=s["info"])
    if op == "trees":
        abg.tree_plan(s["parent"], s["lens"], s["cu"], s["mask"], s["pos"])
        return s["mask"], s["pos"]
    if op == "put":
        if s["case"]["copy"]:
            abg.kv_put(s["k"], s["v"], s["Kc"], s["Vc"], slots=s["slots"], rows=s["rows"])
            return s["Kc"], s["Vc"]
        abg.kv_put(s["k"], s["v"], s["Kc"], s["Vc"], slots=s["slots"], q=s["q"], qo=s["qo"], qn_w=s.get("qn_w"),
                   kn_w=s.get("kn_w"), cos=s["cos"], sin=s["sin"], pos=s["pos"], eps=EPS)
        return s["Kc"], s["Vc"], s["qo"]
    if "ws" not in s:
        s["ws"] = torch.empty(abg.tree_accept_workspace(s["logits"]), dtype=torch.uint8, device="cuda")
    abg.tree_accept(s["logits"], s["tok"], s["parent"], s["cu"], s["best"], s["rows"], s["add"], s["last"], ws=s["ws"])
    return dict(best=s["best"], rows=s["rows"], add=s["add"], last=s["last"])


# -------------------------------------------------------------- 64 bits ----
def exact(c, seed):
    if c["op"] not in ("attn", "put"):
        return None  # whole numbers only
    s = prepare(c, seed)
    if c["op"] == "put":
        k, v = s["k"].double(), s["v"].double()
        out = []
        if c["copy"]:
            k, v = k[s["rows"].long()], v[s["rows"].long()]
        else:
            ang = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()][:, None]

            def turned(x, w):
                if w is not None:
                    x = x * torch.rsqrt((x * x).sum(2, keepdim=True) / x.shape[2] + EPS) * w.double()
                h = x.shape[2] // 2
                z = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous()) * ang
                return torch.cat([z.real, z.imag], 2)

            k = turned(k, s.get("kn_w"))
            out = [turned(s["q"].double(), s.get("qn_w"))]
        page = s["Kc"].shape[2]
        slots = range(c["N"]) if s["slots"] is None else s["slots"].tolist()
        flat = [x.double().transpose(1, 2).reshape(-1, *k.shape[1:]) for x in (s["Kc"], s["Vc"])]
        to = torch.tensor([t for t in slots if t >= 0], device="cuda", dtype=torch.long)
        src = torch.tensor([n for n, t in enumerate(slots) if t >= 0], device="cuda", dtype=torch.long)
        flat[0][to], flat[1][to] = k[src], v[src]
        return tuple([x.view(-1, page, *k.shape[1:]).transpose(1, 2) for x in flat] + out)
    Hkv, page, D = s["Kc"].shape[1:]
    N, Hq = s["q"].shape[:2]
    y = torch.zeros((N, Hq, D), dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    bits = (s["mask"][:, :, None] >> torch.arange(64, device="cuda") & 1).view(N, -1).bool()
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        pages = s["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            K = torch.cat([s["Kc"][pages, h].reshape(-1, D)[:n], s["Kd"][h, lo:hi]]).double()
            V = torch.cat([s["Vc"][pages, h].reshape(-1, D)[:n], s["Vd"][h, lo:hi]]).double()
            for t in range(lo, hi):
                heads = slice(h * Hq // Hkv, (h + 1) * Hq // Hkv)
                a = s["q"][t, heads].double() @ K.T / math.sqrt(D)
                a[:, n:][:, ~bits[t, :hi - lo]] = -math.inf
                y[t, heads] = torch.softmax(a, 1) @ V
    if s["gate"] is not None:
        y = y * torch.sigmoid(s["gate"].double())
    return y if s["ysum"] is None else (y, y.reshape(N, -1, 64).sum(2))
