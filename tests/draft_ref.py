"""Plain 64-bit and integer forms of the draft-verification calls, written from
their definitions in include/abg.h with one loop per request and draft."""
from __future__ import annotations

import numpy as np


def page_plan(lens, add, cu, held, ends, ring, table, page, N):
    table, ring = table.copy(), ring.copy()
    slots, pos = np.full(N, -1, np.int64), np.zeros(N, np.int32)
    lens_out, held_out = lens.copy(), held.copy()
    head, tail = (int(v) for v in ends)
    R, width = len(ring), table.shape[1]
    old = ring.copy()
    asked = taken = freed = refused = 0
    for b in range(len(lens)):
        span = int(cu[b + 1]) - int(cu[b])
        if add[b] < 0:
            if lens[b] < 0 or not 0 <= held[b] <= width:
                refused += 1
                continue
            for j in range(held[b]):
                ring[(tail + freed + j) % R] = table[b, j]
            freed += int(held[b])
            lens_out[b] = held_out[b] = 0
            continue
        total = int(lens[b]) + int(add[b])
        need = -(-total // page)
        if lens[b] < 0 or not 0 <= held[b] <= width or add[b] > span or need > width or total > 2**31 - 1:
            refused += 1
            continue
        extra = max(0, need - int(held[b]))
        asked += extra
        if extra and asked > min(max(tail - head, 0), R):
            refused += 1
            continue
        for j in range(extra):
            table[b, held[b] + j] = old[(head + asked - extra + j) % R]
        taken = asked if extra else taken
        lens_out[b], held_out[b] = total, held[b] + extra
        for i in range(add[b]):
            p = int(lens[b]) + i
            slots[cu[b] + i] = int(table[b, p // page]) * page + p % page
            pos[cu[b] + i] = p
    return dict(slots=slots, pos=pos, table=table, ring=ring, lens=lens_out, held=held_out,
                ends=np.array([head + taken, tail + freed]), info=np.array([taken, refused]))


def tree_plan(parent, lens, cu, words):
    N = len(parent)
    bits, pos = np.zeros((N, 64 * words), bool), np.zeros(N, np.int32)
    for b in range(len(lens)):
        T = min(int(cu[b + 1]) - int(cu[b]), 64 * words)
        p = parent[cu[b]:cu[b] + T]
        for i in range(T):
            if p[i] < -1:
                continue
            at, seen = i, set()
            while at not in seen:
                seen.add(at)
                up = int(p[at])
                if up < 0 or up >= T or up == at or p[up] < -1:
                    break
                at = up
            bits[cu[b] + i, list(seen)] = True
            pos[cu[b] + i] = lens[b] + len(seen) - 1
    return pack(bits), pos


def pack(bits):
    """Bit rows [N][64*words] as int64 words."""
    b = np.packbits(bits, axis=1, bitorder="little")
    return np.ascontiguousarray(b).view(np.int64)


def kv_put(x, w, cos, sin, pos, eps):
    """Norm and rotation of x [N][H][D] in 64 bits."""
    x = x.astype(np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * w.astype(np.float64)
    if cos is not None:
        h = x.shape[2] // 2
        c, s = cos[pos][:, None].astype(np.float64), sin[pos][:, None].astype(np.float64)
        x = np.concatenate([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], 2)
    return x


def tree_attn(q, Kc, Vc, table, lens, cu, Kd, Vd, bits, gate=None):
    """(y [N][Hq][D], terms [N][Hq][2]): the attention in 64 bits, and of each
    row the largest |V| that it sees and the largest sum of |q_i k_i| / sqrt(D)
    (for the error bounds).  All arrays 64-bit; bits [N][64*words]."""
    N, Hq, D = q.shape
    pages, Hkv, page = Kc.shape[:3]
    y, terms = np.zeros((N, Hq, D)), np.zeros((N, Hq, 2))
    cap = bits.shape[1]
    for b in range(len(lens)):
        n = max(0, min(int(lens[b]), table.shape[1] * page))
        lo, T = int(cu[b]), min(int(cu[b + 1]) - int(cu[b]), cap)
        t = np.arange(n)
        ids = table[b, t // page]
        ok = (ids >= 0) & (ids < pages)
        for h in range(Hkv):
            K, V = np.zeros((n, D)), np.zeros((n, D))
            K[ok], V[ok] = Kc[ids[ok], h, t[ok] % page], Vc[ids[ok], h, t[ok] % page]
            for i in range(T):
                see = np.nonzero(bits[lo + i, :T])[0]
                k, v = np.concatenate([K, Kd[h, lo + see]]), np.concatenate([V, Vd[h, lo + see]])
                if not len(k):
                    continue
                for hq in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                    s = k @ q[lo + i, hq] / np.sqrt(D)
                    m = s.max()
                    if m == -np.inf:
                        continue
                    p = np.exp(s - m)
                    with np.errstate(invalid="ignore"):
                        y[lo + i, hq] = p @ v / p.sum()
                    terms[lo + i, hq] = np.abs(v).max(), (np.abs(k) @ np.abs(q[lo + i, hq])).max() / np.sqrt(D)
    if gate is not None:
        y = y / (1.0 + np.exp(-gate))
    return y, terms


def tree_accept(logits, tok, parent, cu, cap=256):
    x = np.where(np.isnan(logits), -np.inf, logits)
    best = x.argmax(1).astype(np.int32)
    rows = np.full(len(tok), -1, np.int32)
    add, last = np.zeros(len(cu) - 1, np.int32), np.full(len(cu) - 1, -1, np.int32)
    for b in range(len(cu) - 1):
        lo, T = int(cu[b]), min(int(cu[b + 1]) - int(cu[b]), cap)
        path, at = [], 0 if T else None
        while at is not None:
            path.append(at)
            at = next((i for i in range(at + 1, T) if parent[lo + i] == at and tok[lo + i] == best[lo + at]), None)
        rows[lo:lo + len(path)] = [lo + i for i in path]
        add[b] = len(path)
        if path:
            last[b] = best[lo + path[-1]]
    return best, rows, add, last
