"""Plain forms of the quantised cache's format, from its definition in
include/abg.h: binary32 steps one by one (numpy rounds each once), and the
values that codes and factors stand for in 64 bits."""
from __future__ import annotations

import numpy as np

F = np.float32


def rows(x, w, cos, sin, pos, eps):
    """Norm (squares summed as the pairwise tree) and rotation of float32 x
    [N][H][D], step by step."""
    x = x.astype(F)
    if w is not None:
        ss = x * x
        while ss.shape[2] > 1:
            ss = ss[..., 0::2] + ss[..., 1::2]
        x = (x * (F(1) / np.sqrt(ss / F(x.shape[2]) + F(eps)))) * w
    if cos is not None:
        ok = (pos >= 0) & (pos < len(cos))
        at = np.where(ok, pos, 0)
        c, s = (np.where(ok[:, None], t[at], F(np.nan))[:, None] for t in (cos, sin))
        a, b = x[..., :x.shape[2] // 2], x[..., x.shape[2] // 2:]
        x = np.concatenate([a * c - b * s, b * c + a * s], 2)
    assert x.dtype == F
    return x


def quantise(x, bits, group):
    """Words [..][D*bits/32] (uint32) and pairs [..][D/group][2] (float16) of
    float32 x [..][D]."""
    x = x.astype(F).reshape(*x.shape[:-1], -1, group)
    bad = ~(np.abs(x) <= F(65504)).all(-1, keepdims=True)
    x = np.where(bad, F(0), x)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    levels = F(2**bits - 1)
    bias, scale = lo.astype(np.float16), ((hi - lo) / levels).astype(np.float16)
    with np.errstate(divide="ignore"):
        inv = np.where(scale > 0, F(1) / scale.astype(F), F(0))
    with np.errstate(invalid="ignore"):
        code = np.clip(np.rint((x - bias.astype(F)) * inv), 0, levels).astype(np.uint32)
    nan = np.array(0x7FFF, np.uint16).view(np.float16)
    pairs = np.where(bad, nan, np.concatenate([scale, bias], -1))
    return pack(code.reshape(*code.shape[:-2], -1), bits), pairs


def pack(code, bits):
    per = 32 // bits
    code = code.reshape(*code.shape[:-1], -1, per).astype(np.uint32)
    return np.bitwise_or.reduce(code << (bits * np.arange(per, dtype=np.uint32)), axis=-1)


def codes(words, bits):
    per = 32 // bits
    c = words.view(np.uint32)[..., None] >> (bits * np.arange(per, dtype=np.uint32)) & np.uint32(2**bits - 1)
    return c.reshape(*words.shape[:-1], -1)


def values(words, pairs, bits):
    """What words and pairs stand for, in 64 bits, and the magnitudes |scale| *
    code + |bias| (for the error bounds)."""
    c = codes(words, bits).astype(np.float64)
    p = np.repeat(pairs.astype(np.float64), c.shape[-1] // pairs.shape[-2], axis=-2)
    return p[..., 0] * c + p[..., 1], np.abs(p[..., 0]) * c + np.abs(p[..., 1])
