"""Cases that time the quantised key-value cache's operators, with their plain forms.

A decoder whose cache is kept in 4 or 8 bits runs `kvq_put` (norm, rotation and
quantisation of the rows that enter the cache), `kvq_attn` (attention of new
tokens, one a request or a tree of drafts, over the quantised pages) and
`kvq_get` (rows of the cache read back, for what wants them in 16 or 32 bits).

The format is the one of this repository's weights, a row of a key/value head
at a time: value = scale * code + bias, codes packed low first into 32-bit
words, one float16 pair (scale, bias) for every 32 or 64 columns.  Of the
float32 values x of a group, each step rounded once:

    bias  = f16(min x),  scale = f16((max x - min x) / (2^bits - 1)),
    code  = clamp(round((x - bias) * (1 / scale)), 0, 2^bits - 1)   (0 where scale is 0).

Head counts and widths are those of this repository's mixer tests and synthetic
decode token; the rest is generic.
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
        # one sequence, one token: latency
        dict(name="attn one token f32 q4", op="attn", type="f32", bits=4, group=64, B=1, T=1, Hq=8, Hkv=2, D=256, L=2047,
             ragged=0.0, page=64, gate=True),
        # a serving batch, one new token each, over long ragged sequences in small pages
        dict(name="attn batch bf16 q4", op="attn", type="bf16", bits=4, group=64, B=64, T=1, Hq=16, Hkv=4, D=128, L=16000,
             ragged=0.5, page=16, gate=False),
        # the same in 8 bits, wider heads
        dict(name="attn batch bf16 q8", op="attn", type="bf16", bits=8, group=64, B=48, T=1, Hq=8, Hkv=2, D=256, L=9001,
             ragged=0.5, page=32, gate=True),
        # one very long sequence, one token
        dict(name="attn long f16 q8", op="attn", type="f16", bits=8, group=32, B=1, T=1, Hq=16, Hkv=2, D=128, L=131071,
             ragged=0.0, page=128, gate=False),
        # a few sequences of drafts (one batched product)
        dict(name="attn drafts f32 q4", op="attn", type="f32", bits=4, group=32, B=4, T=8, Hq=16, Hkv=4, D=128, L=4100,
             ragged=0.5, page=100, gate=True),
        # drafts of a batch: trees of four tokens a sequence
        dict(name="attn trees bf16 q4", op="attn", type="bf16", bits=4, group=64, B=32, T=4, Hq=16, Hkv=2, D=128, L=12000,
             ragged=0.5, page=16, gate=False),
        # the new tokens of a decode step enter the cache (and are read back): latency
        dict(name="put step q4", op="put", type="f32", bits=4, group=64, N=32, Hq=8, Hkv=2, D=256, page=64, copy=False),
        # a long prompt enters the cache, and its own attention reads what the cache holds
        dict(name="put prompt q4", op="put", type="bf16", bits=4, group=64, N=8191, Hq=16, Hkv=4, D=128, page=16,
             copy=False),
        # accepted drafts out of their 16-bit buffers
        dict(name="put drafts q8", op="put", type="bf16", bits=8, group=32, N=777, Hq=16, Hkv=4, D=64, page=16, copy=True),
        # a shared prefix read back for a prompt's attention
        dict(name="get prefix q4", op="get", type="bf16", bits=4, group=64, N=32768, Hkv=4, D=128, page=16),
        # some rows in full, and as many as a short prompt has
        dict(name="get rows q8", op="get", type="f32", bits=8, group=32, N=300, Hkv=2, D=256, page=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "put", "get"])
    bits, group = rng.choice([4, 8]), rng.choice([32, 64])
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 256])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "attn":
        c = dict(op=op, type=kind, bits=bits, group=group, B=_log(rng, 1, 64), T=rng.choice([1, 1, 1, 2, 3, 5, 8]), Hq=Hq,
                 Hkv=Hkv, D=D, L=_log(rng, 16, 131071), ragged=rng.choice([0.0, 0.5, 0.9]),
                 page=rng.choice([16, 32, 64, 100, 128]), gate=rng.random() < 0.5)
        while True:  # no more than the largest listed ones read and compute
            w = work(c)
            if w["bytes"] <= 3.5e8 and w["flops"] <= (2e9 if kind == "f32" else 2e10) and \
                    c["B"] * Hkv * D * c["L"] <= 4e8:
                return c
            if c["L"] > 512:
                c["L"] = c["L"] * 2 // 3
            else:
                c["B"] = max(1, c["B"] // 2)
    if op == "put":
        return dict(op=op, type=kind, bits=bits, group=group, N=_log(rng, 1, 4000), Hq=Hq, Hkv=Hkv, D=D,
                    page=rng.choice([16, 32, 100]), copy=rng.random() < 0.3)
    return dict(op=op, type=kind, bits=bits, group=group, N=_log(rng, 1, 15000), Hkv=Hkv, D=D, page=rng.choice([16, 32, 100]))


# ----------------------------------------------------------------- sizes ----
def _lens(c):
    """Cached tokens of each sequence (a fixed ragged pattern of the case)."""
    return [int(round(c["L"] * (1.0 - c["ragged"] * ((b + 1) * 0.6180339887 % 1.0)))) for b in range(c["B"])]


def _row_bytes(c):
    """Bytes of one head's row of K (or V) in the cache."""
    return c["D"] * c["bits"] // 8 + 4 * c["D"] // c["group"]


def work(c):
    e, D = (4 if c["type"] == "f32" else 2), c["D"]
    if c["op"] == "attn":
        lens, T, Hq = _lens(c), c["T"], c["Hq"]
        N = c["B"] * T
        io = N * Hq * D * (2 * e + (4 if c["gate"] else 0)) + 2 * c["Hkv"] * D * e * N + 8 * N
        return {"bytes": 2 * c["Hkv"] * _row_bytes(c) * sum(lens) + io,
                "flops": 4 * D * Hq * sum(T * (n + (T + 1) / 2) for n in lens)}
    cached = 2 * c["N"] * c["Hkv"] * _row_bytes(c)
    back = cached + c["N"] * (8 + 2 * c["Hkv"] * D * e)  # the reading
    if c["op"] == "get":
        return {"bytes": back, "flops": 2 * 2 * c["N"] * c["Hkv"] * D}
    if c["copy"]:
        return {"bytes": back + cached + c["N"] * (12 + 2 * c["Hkv"] * D * e), "flops": 10 * c["N"] * c["Hkv"] * D}
    rows = c["N"] * (12 + 4 * D + (c["Hq"] + 2 * c["Hkv"]) * D * 4 + c["Hq"] * D * e)
    return {"bytes": back + cached + rows, "flops": c["N"] * D * (10 * c["Hkv"] + 9 * (c["Hq"] + c["Hkv"]))}


# ---------------------------------------------------------------- inputs ----
def _i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


def _parents(rng, spans):
    """Local parent index of each draft: node 0 is the root, later ones hang off
    one of the eight before them."""
    return np.concatenate([[-1 if i == 0 else int(rng.integers(max(0, i - 8), i)) for i in range(t)] for t in spans])


def _ancestors(parent, spans):
    """Mask words [N][1]: bit j of a node says that it is j or below j."""
    out = np.zeros((len(parent), 1), np.uint64)
    at = 0
    for t in spans:
        for i in range(t):
            p = parent[at + i]
            out[at + i] = (out[at + p] if p >= 0 else 0) | np.uint64(1 << i)
        at += t
    return torch.from_numpy(out.view(np.int64)).cuda()


def _pack(code, bits):
    """Codes [...][D] (int32) as words [...][D*bits/32], low columns first."""
    per = 32 // bits
    code = code.view(*code.shape[:-1], code.shape[-1] // per, per)
    word = code[..., 0].clone()
    for i in range(1, per):
        word |= code[..., i] << (bits * i)
    return word


def _cache(shape, bits, group, normal):
    """Words and factors of quantised normal rows [pages][Hkv][page][D]."""
    words = torch.empty((*shape[:-1], shape[-1] * bits // 32), dtype=torch.int32, device="cuda")
    pairs = torch.empty((*shape[:-1], shape[-1] // group, 2), dtype=torch.float16, device="cuda")
    step = max(1, (1 << 26) // int(np.prod(shape[1:])))
    for i in range(0, shape[0], step):
        part = words[i:i + step].shape[0]
        # columns of different sizes, as keys and values have them
        x = normal(part, *shape[1:]) * torch.linspace(0.5, 1.5, shape[-1], device="cuda")
        code, pair = _quantised(x, bits, group)
        words[i:i + step], pairs[i:i + step] = _pack(code.int(), bits), pair
    return words, pairs


def prepare(c, seed):
    rng = np.random.default_rng([seed, 23])
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)

    T, D, Hkv, page, bits, group = TYPES[c["type"]], c["D"], c["Hkv"], c["page"], c["bits"], c["group"]
    s = dict(case=c, op=c["op"])

    def cache(pages):
        shape = (pages, Hkv, page, D)
        return (*_cache(shape, bits, group, normal), *_cache(shape, bits, group, normal))

    if c["op"] == "attn":
        B, Hq = c["B"], c["Hq"]
        lens, spans = _lens(c), [c["T"]] * c["B"]
        N = sum(spans)
        counts = [-(-n // page) for n in lens]
        pages, width = sum(counts) + 3, max(1, max(counts))
        order = rng.permutation(pages)
        table = np.full((B, width), -1)
        at = 0
        for b, n in enumerate(counts):
            table[b, :n] = order[at:at + n]
            at += n
        s.update(cache=cache(pages), q=normal(N, Hq, D, scale=1.5, dtype=T), Kd=normal(Hkv, N, D, dtype=T),
                 Vd=normal(Hkv, N, D, dtype=T), gate=normal(N, Hq, D) if c["gate"] else None, table=_i32(table),
                 lens=_i32(lens), cu=_i32(c["T"] * np.arange(B + 1)), mask=_ancestors(_parents(rng, spans), spans),
                 max_len=max(lens), max_span=c["T"], y=torch.empty((N, Hq, D), dtype=T, device="cuda"),
                 ysum=torch.empty((N, Hq * D // 64), device="cuda") if T == torch.float32 else None)
        return s
    N = c["N"]
    pages = -(-N // page) + 2
    order = rng.permutation(pages)
    p = int(rng.integers(0, page)) + np.arange(N)
    slots = order[p // page] * page + p % page
    s.update(slots=torch.as_tensor(slots, dtype=torch.int64).cuda(), ko=torch.empty((N, Hkv, D), dtype=T, device="cuda"),
             vo=torch.empty((N, Hkv, D), dtype=T, device="cuda"))
    if c["op"] == "get":
        s["cache"] = cache(pages)
        return s
    words = lambda: torch.zeros((pages, Hkv, page, D * bits // 32), dtype=torch.int32, device="cuda")  # noqa: E731
    pairs = lambda: torch.zeros((pages, Hkv, page, D // group, 2), dtype=torch.float16, device="cuda")  # noqa: E731
    s["cache"] = (words(), pairs(), words(), pairs())
    if c["copy"]:
        rows = np.sort(rng.permutation(2 * N)[:N])
        s.update(k=normal(Hkv, 2 * N, D, dtype=T).transpose(0, 1), v=normal(Hkv, 2 * N, D, dtype=T).transpose(0, 1),
                 rows=_i32(rows))
        return s
    Hq = c["Hq"]
    qkv = normal(N, Hq + 2 * Hkv, D, scale=1.5)  # one product's output
    ang = torch.rand((N + 999, D // 2), device="cuda", generator=gen) * (2 * math.pi)
    s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], cos=ang.cos(), sin=ang.sin(),
             pos=_i32(int(rng.integers(0, 1000)) + np.arange(N)), qo=torch.empty((N, Hq, D), dtype=T, device="cuda"),
             qn_w=1 + normal(D, scale=0.1), kn_w=1 + normal(D, scale=0.1))
    return s


# ------------------------------------------------------------ plain forms ----
def _quantised(x, bits, group):
    """Codes [...][D] and pairs [...][D/group][2] of float32 rows, each step rounded once."""
    g = x.view(*x.shape[:-1], x.shape[-1] // group, group)
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    levels = torch.full((1,), 2.0**bits - 1, device=x.device)  # (a tensor: a division, not a product)
    bias, scale = lo.half(), ((hi - lo) / levels).half()
    inv = torch.where(scale > 0, 1.0 / scale.float(), 0.0)
    code = ((g - bias.float()) * inv).round().clamp(0, 2**bits - 1)
    return code.view(x.shape), torch.cat([scale, bias], -1)


def _values(words, pairs, bits):
    """What words [...][D*bits/32] and pairs [...][D/group][2] stand for, float32."""
    code = (words.unsqueeze(-1) >> (bits * torch.arange(32 // bits, device="cuda", dtype=torch.int32))) & (2**bits - 1)
    G = pairs.shape[-2]
    code = code.view(*words.shape[:-1], G, words.shape[-1] * (32 // bits) // G).float()
    pairs = pairs.float()
    return (code * pairs[..., :1] + pairs[..., 1:]).flatten(-2)


def _padded(s):
    """Row of draft t of request b [B][T]."""
    return s["cu"][:-1, None].long() + torch.arange(s["max_span"], device="cuda")


def _plain_attn(s):
    Kc, Ks, Vc, Vs = s["cache"]
    bits, Hkv, page, D = s["case"]["bits"], s["case"]["Hkv"], s["case"]["page"], s["case"]["D"]
    N, Hq = s["q"].shape[:2]
    B, L, G = len(s["lens"]), s["max_len"], Hq // Hkv
    idx = _padded(s)
    T = idx.shape[1]
    at = torch.arange(L, device="cuda")
    pages, row = s["table"].long().clamp(min=0)[:, at // page], (at % page)[None]
    K = _values(Kc[pages, :, row], Ks[pages, :, row], bits).permute(0, 2, 1, 3)
    Kd, Vd = (s[n][:, idx].transpose(0, 1).float() for n in ("Kd", "Vd"))
    q = s["q"][idx].float().view(B, T, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, T * G, D)
    sees = (s["mask"][idx] >> torch.arange(T, device="cuda")) & 1 > 0
    sees = sees[:, None, :, None, :].expand(B, 1, T, G, T).reshape(B, 1, T * G, T)
    S = torch.cat([(q @ K.transpose(2, 3)).masked_fill_((at >= s["lens"][:, None])[:, None, None], -math.inf),
                   (q @ Kd.transpose(2, 3)).masked_fill_(~sees, -math.inf)], 3).mul_(D ** -0.5)
    del K
    p = S.sub_(S.amax(3, keepdim=True)).exp_()  # (each token sees itself)
    V = _values(Vc[pages, :, row], Vs[pages, :, row], bits).permute(0, 2, 1, 3)
    o = (p[..., :L] @ V + p[..., L:] @ Vd) / p.sum(3, keepdim=True)
    y = torch.empty((N, Hq, D), device="cuda")
    y[idx] = o.view(B, Hkv, T, G, D).transpose(1, 2).reshape(B, T, Hq, D)
    if s["gate"] is not None:
        y = y * (1.0 / (1.0 + torch.exp(-s["gate"])))
    if s["ysum"] is not None:
        return y, y.view(N, Hq * D // 64, 64).sum(2)
    return y.to(s["q"].dtype)


def _plain_rope(s, x, w):
    """Norm (the squares summed as a pairwise tree) and rotation, each step rounded once."""
    D = x.shape[2]
    ss = x * x
    while ss.shape[2] > 1:
        ss = ss[..., 0::2] + ss[..., 1::2]
    x = x * (1.0 / (ss / D + EPS).sqrt()) * w
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], 2)


def _plain_put(s):
    c = s["case"]
    k, v = s["k"], s["v"]
    if c["copy"]:
        k, v = k[s["rows"].long()].float(), v[s["rows"].long()].float()
    else:
        k = _plain_rope(s, k, s["kn_w"])
    out = []
    for x in (k, v.contiguous()):
        code, pair = _quantised(x, c["bits"], c["group"])
        value = code.view(*code.shape[:-1], -1, c["group"]) * pair[..., :1].float() + pair[..., 1:].float()
        out.append(value.flatten(-2).to(TYPES[c["type"]]))
    return tuple(out) if c["copy"] else (*out, _plain_rope(s, s["q"], s["qn_w"]).to(TYPES[c["type"]]))


def _plain_get(s):
    Kc, Ks, Vc, Vs = s["cache"]
    page, T = s["case"]["page"], TYPES[s["case"]["type"]]
    at, row = s["slots"] // page, s["slots"] % page
    return tuple(_values(w[at, :, row], f[at, :, row], s["case"]["bits"]).to(T) for w, f in ((Kc, Ks), (Vc, Vs)))


# -------------------------------------------------------------- the calls ----
def run(s):
    op = s["op"]
    if not own:
        return {"attn": _plain_attn, "put": _plain_put, "get": _plain_get}[op](s)
    import affine_bit_group_gb300 as abg
    if op == "attn":
        if "ws" not in s:  # kept with the buffers, as a decoding loop does
            s["ws"] = torch.empty(abg.kvq_attn_workspace(s["q"], s["cache"], s["max_span"]), dtype=torch.uint8,
                                  device="cuda")
        abg.kvq_attn(s["q"], s["cache"], s["table"], s["lens"], s["cu"], s["Kd"], s["Vd"], s["mask"], s["y"],
                     max_span=s["max_span"], gate=s["gate"], ysum=s["ysum"], ws=s["ws"])
        return s["y"] if s["ysum"] is None else (s["y"], s["ysum"])
    if op == "get":
        abg.kvq_get(s["cache"], s["ko"], s["vo"], slots=s["slots"])
        return s["ko"], s["vo"]
    if s["case"]["copy"]:
        abg.kvq_put(s["k"], s["v"], s["cache"], slots=s["slots"], rows=s["rows"])
    else:
        abg.kvq_put(s["k"], s["v"], s["cache"], slots=s["slots"], q=s["q"], qo=s["qo"], qn_w=s["qn_w"], kn_w=s["kn_w"],
                    cos=s["cos"], sin=s["sin"], pos=s["pos"], eps=EPS)
    abg.kvq_get(s["cache"], s["ko"], s["vo"], slots=s["slots"])
    return (s["ko"], s["vo"]) if s["case"]["copy"] else (s["ko"], s["vo"], s["qo"])


# -------------------------------------------------------------- 64 bits ----
def _rounded(x):
    """64-bit values rounded to 32 bits."""
    return x.float().double()


def _held(x, bits, group):
    """What the cache holds of 32-bit values x (given in 64 bits): the format's roundings done one by one on 64-bit
    values (which a step's exact result, or one rounded to 53 bits, rounds to the same 32 bits)."""
    rows = x.reshape(-1, group)
    low, high = rows.min(1).values, rows.max(1).values
    b = low.float().half().double()
    d = _rounded(_rounded(high - low) / (2**bits - 1)).half().double()
    code = torch.zeros_like(rows)
    there = d > 0
    r = _rounded(1.0 / d[there])
    code[there] = torch.round(_rounded(_rounded(rows[there] - b[there, None]) * r[:, None])).clamp(0, 2**bits - 1)
    return (b[:, None] + d[:, None] * code).view(x.shape)


def _read(words, pairs, pages, rows, bits):
    """Rows of the cache in 64 bits: words[pages, :, rows]."""
    w = words[pages, :, rows].contiguous().view(torch.uint8)
    code = w if bits == 8 else torch.stack([w & 15, w >> 4], -1).flatten(-2)
    f = pairs[pages, :, rows].double().repeat_interleave(code.shape[-1] // pairs.shape[-2], dim=-2)
    return code.double() * f[..., 0] + f[..., 1]


def exact(c, seed):
    s = prepare(c, seed)
    D, page, bits, group = c["D"], c["page"], c["bits"], c["group"]
    if c["op"] == "get":
        Kc, Ks, Vc, Vs = s["cache"]
        return tuple(_read(w, f, s["slots"] // page, s["slots"] % page, bits) for w, f in ((Kc, Ks), (Vc, Vs)))
    if c["op"] == "put":
        k, v = s["k"].double(), s["v"].double()
        if c["copy"]:
            return tuple(_held(x[s["rows"].long()], bits, group) for x in (k, v))
        ang = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()][:, None]
        h = D // 2
        # the key's 32-bit steps, which decide the codes
        t = _rounded(k * k)
        while t.shape[2] > 1:
            t = _rounded(t.unflatten(2, (-1, 2)).sum(3))
        t = _rounded(1.0 / _rounded(_rounded(_rounded(t / D) + torch.tensor(EPS).double()).sqrt()))
        k = _rounded(_rounded(k * t) * s["kn_w"].double())
        a, b, cs, sn = k[..., :h], k[..., h:], ang.real, ang.imag
        k = torch.cat([_rounded(_rounded(a * cs) - _rounded(b * sn)), _rounded(_rounded(b * cs) + _rounded(a * sn))], 2)
        q = s["q"].double()
        q = q * torch.rsqrt((q * q).sum(2, keepdim=True) / D + EPS) * s["qn_w"].double()
        z = torch.complex(q[..., :h].contiguous(), q[..., h:].contiguous()) * ang
        return _held(k, bits, group), _held(v, bits, group), torch.cat([z.real, z.imag], 2)
    Kc, Ks, Vc, Vs = s["cache"]
    N, Hq = s["q"].shape[:2]
    G = Hq // c["Hkv"]
    y = torch.zeros((N, Hq, D), dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    seen = (s["mask"] >> torch.arange(64, device="cuda") & 1).bool()
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        t = torch.arange(n, device="cuda")
        at = s["table"][b].long()[t // page]
        K = torch.cat([_read(Kc, Ks, at, t % page, bits), s["Kd"][:, lo:hi].transpose(0, 1).double()])
        V = torch.cat([_read(Vc, Vs, at, t % page, bits), s["Vd"][:, lo:hi].transpose(0, 1).double()])
        q = s["q"][lo:hi].double().view(hi - lo, c["Hkv"], G, D)
        a = torch.einsum("thgd,nhd->thgn", q, K) / math.sqrt(D)
        a[..., n:] = torch.where(seen[lo:hi, None, None, :hi - lo], a[..., n:], -math.inf)
        y[lo:hi] = torch.einsum("thgn,nhd->thgd", torch.softmax(a, 3), V).reshape(hi - lo, Hq, D)
    if s["gate"] is not None:
        y = y * torch.sigmoid(s["gate"].double())
    return y if s["ysum"] is None else (y, y.reshape(N, -1, 64).sum(2))
