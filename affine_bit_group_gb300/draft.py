"""Decoding several requests with drafted tokens over a paged cache.

The synthetic decoder of `decode` with the attention it leaves out: per layer

    rmsq(h) -> {q, k, v} products -> kv_put (norm, rotation, the drafts' rows)
    -> tree_attn over the request's pages and the drafts -> o product
    -> rmsq -> {gate, up} products -> swq -> down product (the next h)

then the final rmsq, the output head, `tree_accept`, and, for the drafts that
the logits agree with, `page_plan` and a `kv_put` per layer into the pages.  A
request's first draft is its last known token, so that every step accepts at
least one; a step whose trees are single tokens is ordinary decoding.

With a cache in 4 or 8 bits, kvq_put and kvq_attn take the places of kv_put and
tree_attn.  The drafts' rows are then quantised and read back (kvq_get) before
the attention, so that a draft sees the others as it would see them in the cache,
and a step of several drafts gives what as many steps of one give.  The accepted
ones are quantised into the cache from the same products again, since rows that
were read back need not have the codes that they came from (of a group far from 0
the bias's rounding is many scales).

All of a step's calls are queued on the current stream; nothing is read back
between them.  The products take up to eight tokens at a time (abg_q4mm).
"""
from __future__ import annotations

import torch

from . import (MAX_SPAN, kv_put, kvq_attn, kvq_attn_workspace, kvq_cache, kvq_get, kvq_put, page_plan, q4mm,
               rmsq, swq, tree_accept, tree_attn, tree_attn_workspace, tree_plan)

Q4MM_TOKENS = 8  # abg_q4mm's most
QUANTISED = {"q4": 4, "q8": 8}  # bits


def rotation(positions: int, D: int, base: float = 10000.0):
    """cos, sin [positions][D/2] of pos / base^(2i/D)."""
    ang = torch.arange(positions, dtype=torch.float64)[:, None] / base ** (torch.arange(0, D, 2, dtype=torch.float64) / D)
    return ang.cos().float().cuda(), ang.sin().float().cuda()


class DraftDecoder:
    """A decoder's state for `requests` requests: a paged cache of `pages` pages
    of `page` tokens in `cache` (float32, bfloat16, float16, or "q4" or "q8": 4 or
    8 bits in groups of `group` columns), up to max_len tokens (whole pages) a
    request, and the buffers of a step of at most `rows` drafts.

    dm: the weights (decode.DeviceModel), q_rows = Hq*D and kv_rows = Hkv*D;
    embed: [vocabulary][hidden] float32; qn_w, kn_w: [D] norm weights of q and k
    (default 1).
    """

    def __init__(self, dm, embed, D: int, requests: int, pages: int, page: int = 16, max_len: int = 4096,
                 rows: int = 64, cache=torch.float32, eps: float = 1e-6, qn_w=None, kn_w=None, group: int = 64):
        self.dm, self.embed, self.D, self.page, self.eps, self.rows = dm, embed, D, page, eps, rows
        L = dm.layers[0]
        self.Hq, self.Hkv = L["q"].rows // D, L["k"].rows // D
        ones = torch.ones(D, device="cuda")
        self.qn_w, self.kn_w = ones if qn_w is None else qn_w, ones if kn_w is None else kn_w
        width = -(-max_len // page)
        self.cos, self.sin = rotation(width * page, D)  # a position for every token that the table holds
        self.quantised = cache in QUANTISED
        self.ty = torch.float32 if self.quantised else cache  # of the drafts' rows
        if self.quantised:
            bits = QUANTISED[cache]
            self.caches = [kvq_cache(pages, self.Hkv, page, D, bits, group) for _ in dm.layers]
            self.drafts = kvq_cache(1, self.Hkv, rows, D, bits, group)  # of one layer at a time
        else:
            kv = (len(dm.layers), pages, self.Hkv, page, D)
            self.Kc, self.Vc = torch.zeros(kv, dtype=cache, device="cuda"), torch.zeros(kv, dtype=cache, device="cuda")
        kv = (1 if self.quantised else len(dm.layers), self.Hkv, rows, D)
        self.Kd, self.Vd = torch.zeros(kv, dtype=self.ty, device="cuda"), torch.zeros(kv, dtype=self.ty, device="cuda")

        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device="cuda")

        # two copies of what a plan reads and writes
        self.lens, self.held = [i32(requests), i32(requests)], [i32(requests), i32(requests)]
        self.ends = [torch.tensor([0, pages], device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")]
        self.ring = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.table = i32(requests, width)
        self.info, self.last, self.add = i32(2), i32(requests), i32(requests)

    def _products(self, ms, x, xs):
        """x [N][cols] times each matrix."""
        out = [torch.empty((len(x), m.rows), device="cuda") for m in ms]
        for i in range(0, len(x), Q4MM_TOKENS):
            part = slice(i, i + Q4MM_TOKENS)
            for m, y in zip(ms, out):
                q4mm(m.w, m.scale, m.bias, x[part], xs[part], y[part], m.cols)
        return out

    def _norm(self, h, wt):
        xn, xs = torch.empty_like(h), torch.empty((len(h), h.shape[1] // 64), device="cuda")
        for n in range(len(h)):
            rmsq(h[n], wt, xn[n], xs[n], eps=self.eps)
        return xn, xs

    def _plan(self, add, cu, N):
        """page_plan for this step; the next step reads what it wrote."""
        slots, pos = torch.empty(N, dtype=torch.int64, device="cuda"), torch.empty(N, dtype=torch.int32, device="cuda")
        page_plan(self.lens[0], add, cu, self.held[0], self.ends[0], self.ring, self.table, self.page, slots, pos,
                  self.lens[1], self.held[1], self.ends[1], self.info)
        for pair in (self.lens, self.held, self.ends):
            pair.reverse()
        return slots

    def release(self, ended):
        """Gives the pages of the requests b with ended[b] back."""
        self._plan(torch.where(ended.cuda(), -1, 0).int(), torch.zeros(len(self.last) + 1, dtype=torch.int32, device="cuda"), 0)

    def logits(self, tok, parent, cu, max_span: int):
        """Logits [N][vocabulary] of the drafts tok [N] (int32) with parents
        parent [N] and spans cu [requests+1]; their key and value rows are left
        in Kd, Vd, or with a quantised cache before norm and rotation in products,
        and their positions in pos."""
        dm, D, Hq, Hkv, N = self.dm, self.D, self.Hq, self.Hkv, len(tok)
        if not 0 < N <= self.rows or not 0 < max_span <= MAX_SPAN:
            raise ValueError(f"1 to {self.rows} drafts, spans of 1 to {MAX_SPAN}")
        words = (max_span + 63) // 64
        mask, pos = torch.empty((N, words), dtype=torch.int64, device="cuda"), torch.empty(N, dtype=torch.int32, device="cuda")
        tree_plan(parent, self.lens[0], cu, mask, pos)
        h = self.embed[tok.long()]
        qo = torch.empty((N, Hq, D), dtype=self.ty, device="cuda")
        y, ysum = torch.empty((N, Hq, D), device="cuda"), torch.empty((N, Hq * D // 64), device="cuda")
        ws = torch.empty(kvq_attn_workspace(qo, self.caches[0], max_span) if self.quantised else
                         tree_attn_workspace(qo, self.Kc[0], max_span), dtype=torch.uint8, device="cuda")
        self.products, self.pos = [], pos
        for i, L in enumerate(dm.layers):
            q, k, v = self._products([L["q"], L["k"], L["v"]], *self._norm(h, L["rms1"]))
            k, v = k.view(N, Hkv, D), v.view(N, Hkv, D)
            rope = dict(q=q.view(N, Hq, D), qo=qo, qn_w=self.qn_w, kn_w=self.kn_w, cos=self.cos, sin=self.sin, pos=pos,
                        eps=self.eps)
            if self.quantised:
                self.products.append((k, v))
                kvq_put(k, v, self.drafts, **rope)
                kvq_get(self.drafts, self.Kd[0, :, :N].transpose(0, 1), self.Vd[0, :, :N].transpose(0, 1))
                kvq_attn(qo, self.caches[i], self.table, self.lens[0], cu, self.Kd[0], self.Vd[0], mask, y,
                         max_span=max_span, ysum=ysum, ws=ws)
            else:
                kv_put(k, v, self.Kd[i].unsqueeze(0), self.Vd[i].unsqueeze(0), **rope)
                tree_attn(qo, self.Kc[i], self.Vc[i], self.table, self.lens[0], cu, self.Kd[i], self.Vd[i], mask, y,
                          max_span=max_span, ysum=ysum, ws=ws)
            o, = self._products([L["o"]], y.view(N, Hq * D), ysum)
            gate, up = self._products([L["gate"], L["up"]], *self._norm(o, L["rms2"]))
            a = torch.cat([gate, up], 1)
            s, ss = torch.empty_like(gate), torch.empty((N, gate.shape[1] // 64), device="cuda")
            for n in range(N):
                swq(a[n], s[n], ss[n])
            h, = self._products([L["down"]], s, ss)
        return self._products([dm.head], *self._norm(h, dm.rms_final))[0]

    def step(self, tok, parent, cu, max_span: int):
        """One step: the drafts' logits, the check, and the accepted drafts' rows
        into the cache.  Returns (rows, add, last): rows[cu[b]+i] is the i-th
        accepted draft of request b, add[b] their number, last[b] the token
        that follows them (all on the GPU).  A request whose accepted drafts
        find no page, or no place in its table row, is refused (info[1] counts
        them): its rows are -1, add[b] is 0 and last[b] is its first draft's
        token, with which it can go on once pages have been given back."""
        N = len(tok)
        best, rows = (torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(2))
        tree_accept(self.logits(tok, parent, cu, max_span), tok, parent, cu, best, rows, self.add, self.last)
        slots = self._plan(self.add, cu, N)
        if self.quantised:
            pos = self.pos[rows.clamp(min=0).long()]
            for (k, v), cache in zip(self.products, self.caches):
                kvq_put(k, v, cache, slots=slots, rows=rows, kn_w=self.kn_w, cos=self.cos, sin=self.sin, pos=pos, eps=self.eps)
        else:
            for i in range(len(self.dm.layers)):
                kv_put(self.Kd[i].transpose(0, 1), self.Vd[i].transpose(0, 1), self.Kc[i], self.Vc[i], slots=slots, rows=rows)
        stored = self.lens[0] - self.lens[1]  # a refused request's length has not changed
        rows.masked_fill_(slots < 0, -1)
        torch.where(stored != self.add, tok[cu[:-1].clamp(max=N - 1).long()], self.last, out=self.last)
        self.add.copy_(stored)
        return rows, self.add, self.last
