"""Refusals of the draft-verification calls, without a GPU: every argument
error that the host can see has its documented status before any device work."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

import affine_bit_group_gb300 as abg
import draft_ref as ref

OK, EINVAL, EALIGN, ESHAPE, EALIAS = 0, 1, 2, 3, 4
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x7F0000000000  # fake device addresses, 16 MB apart
STEP = 1 << 24


@pytest.fixture(scope="module")
def lib():
    return abg.library()


@pytest.mark.parametrize("ctype,cname", [(abg._KvPutArgs, "abg_kv_put_args"), (abg._TreeAttnArgs, "abg_tree_attn_args")])
def test_struct_layout_matches_c(tmp_path, ctype, cname):
    fields = [f for f, _ in ctype._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text("\n".join(
        ["#include <stdio.h>", "#include <stddef.h>", '#include "abg.h"', "int main(void){",
         f'printf("%zu %d %d\\n", sizeof({cname}), ABG_MAX_SPAN, ABG_MAX_REQUESTS);'] +
        [f'printf("%zu\\n", offsetof({cname}, {f}));' for f in fields] + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    out = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert out[:3] == [ctypes.sizeof(ctype), abg.MAX_SPAN, abg.MAX_REQUESTS]
    assert out[3:] == [getattr(ctype, f).offset for f in fields]


PLAN = dict(lens=A, add=A + STEP, cu=A + 2 * STEP, held=A + 3 * STEP, ends=A + 4 * STEP, ring=A + 5 * STEP,
            table=A + 6 * STEP, slots=A + 7 * STEP, pos=A + 8 * STEP, lens_out=A + 9 * STEP, held_out=A + 10 * STEP,
            ends_out=A + 11 * STEP, info=A + 12 * STEP, B=4, N=32, page=16, width=8, ring_len=64)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), ESHAPE), (dict(B=8193), ESHAPE), (dict(N=-1), ESHAPE), (dict(N=2**31), ESHAPE), (dict(page=0), ESHAPE),
    (dict(width=0), ESHAPE), (dict(ring_len=0), ESHAPE), (dict(ring_len=2**31), ESHAPE),
    *[({k: None}, EINVAL) for k in PLAN if k not in ("B", "N", "page", "width", "ring_len")],
    (dict(lens=A + 2), EALIGN), (dict(ends=A + 4 * STEP + 4), EALIGN), (dict(slots=A + 7 * STEP + 4), EALIGN),
    (dict(lens_out=A), EALIAS), (dict(held_out=A + 3 * STEP), EALIAS), (dict(ends_out=A + 4 * STEP), EALIAS),
    (dict(pos=A + 7 * STEP + 8 * 31), EALIAS), (dict(info=A + 6 * STEP + 4 * 31), EALIAS)])
def test_page_plan_refuses(lib, change, status):
    assert lib.abg_page_plan(*{**PLAN, **change}.values(), None) == status


TREE = dict(parent=A, lens=A + STEP, cu=A + 2 * STEP, mask=A + 3 * STEP, pos=A + 4 * STEP, B=3, N=20, words=2)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), ESHAPE), (dict(N=-1), ESHAPE), (dict(words=0), ESHAPE), (dict(words=5), ESHAPE), (dict(N=0), OK),
    *[({k: None}, EINVAL) for k in ("parent", "lens", "cu", "mask", "pos")],
    (dict(mask=A + 3 * STEP + 4), EALIGN), (dict(pos=A + 4 * STEP + 1), EALIGN), (dict(pos=A + 4 * 19), EALIAS),
    (dict(pos=A + 3 * STEP + 16 * 19 + 8), EALIAS)])
def test_tree_plan_refuses(lib, change, status):
    assert lib.abg_tree_plan(*{**TREE, **change}.values(), None) == status


PUT = dict(q=A, k=A + STEP, v=A + 2 * STEP, q_row=512, q_head=128, k_row=256, k_head=128, v_row=256, v_head=128,
           rows=None, slots=A + 3 * STEP, qn_w=A + 4 * STEP, kn_w=A + 5 * STEP, cos=A + 6 * STEP, sin=A + 7 * STEP,
           pos=A + 8 * STEP, qo=A + 9 * STEP, Kc=A + 10 * STEP, Vc=A + 11 * STEP, N=10, src_rows=10, Hq=4, Hkv=2, D=128,
           page=16, pages=8, cos_rows=100, eps=1e-6, src_type=0, type=1)


@pytest.mark.parametrize("change,status", [
    (dict(type=3), EINVAL), (dict(src_type=2), EINVAL), (dict(D=96), ESHAPE), (dict(Hkv=0), ESHAPE),
    (dict(Hq=0), ESHAPE), (dict(page=0), ESHAPE), (dict(pages=-1), ESHAPE), (dict(N=11), ESHAPE),
    (dict(N=-1), ESHAPE), (dict(k_row=-256), ESHAPE), (dict(pages=2**31 - 1, page=2**31 - 1, Hkv=60000), ESHAPE),
    (dict(cos_rows=0), ESHAPE), (dict(N=0), OK), (dict(sin=None), EINVAL), (dict(qo=None), EINVAL),
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(Kc=None), EINVAL),
    (dict(Vc=None), EINVAL), (dict(pos=None), EINVAL), (dict(k=A + STEP + 8), EALIGN), (dict(k_row=257), EALIGN),
    (dict(q_head=126), EALIGN), (dict(slots=A + 3 * STEP + 4), EALIGN), (dict(cos=A + 6 * STEP + 4), EALIGN),
    (dict(Vc=A + 10 * STEP), EALIAS), (dict(qo=A), EALIAS), (dict(Kc=A + STEP + 4 * (256 * 9 + 255) - 12), EALIAS),
    (dict(qo=A + 3 * STEP + 64), EALIAS)])
def test_kv_put_refuses(lib, change, status):
    a = abg._KvPutArgs(**{**PUT, **change})
    assert lib.abg_kv_put(ctypes.byref(a), None) == status
    assert lib.abg_kv_put(None, None) == EINVAL


ATTN = dict(q=A, Kc=A + STEP, Vc=A + 2 * STEP, table=A + 3 * STEP, lens=A + 4 * STEP, cu=A + 5 * STEP, Kd=A + 6 * STEP,
            Vd=A + 7 * STEP, mask=A + 8 * STEP, gate=A + 9 * STEP, y=A + 10 * STEP, ysum=None, B=3, N=20, Hq=8, Hkv=2,
            D=128, page=16, pages=50, width=20, drafts=20, words=1, max_span=8, type=1, y_type=1)
WS = A + 64 * STEP


@pytest.mark.parametrize("change,status", [
    (dict(type=3), EINVAL), (dict(y_type=2), EINVAL), (dict(ysum=A + 11 * STEP), EINVAL), (dict(words=0), ESHAPE),
    (dict(words=5), ESHAPE), (dict(B=0), ESHAPE), (dict(N=-1), ESHAPE), (dict(N=0), OK), (dict(D=80), ESHAPE),
    (dict(Hq=7), ESHAPE), (dict(Hkv=0), ESHAPE), (dict(Hq=1, Hkv=2), ESHAPE), (dict(page=0), ESHAPE),
    (dict(drafts=19), ESHAPE), (dict(max_span=0), ESHAPE), (dict(max_span=65), ESHAPE),
    (dict(width=2**20, page=2**12), ESHAPE), *[({k: None}, EINVAL) for k in (
        "q", "Kc", "Vc", "table", "lens", "cu", "Kd", "Vd", "mask", "y")],
    (dict(table=None, pages=0), EINVAL), (dict(q=A + 8), EALIGN), (dict(gate=A + 9 * STEP + 4), EALIGN),
    (dict(mask=A + 8 * STEP + 4), EALIGN), (dict(y=A), EALIAS), (dict(y=A + 9 * STEP), EALIAS),
    (dict(y=WS), EALIAS), (dict(y_type=0, ysum=A + 10 * STEP), EALIAS)])
def test_tree_attn_refuses(lib, change, status):
    a = abg._TreeAttnArgs(**{**ATTN, **change})
    assert lib.abg_tree_attn(ctypes.byref(a), WS, 1 << 40, None) == status


def test_tree_attn_workspace_is_asked_for(lib):
    n = ctypes.c_int64()
    assert lib.abg_tree_attn_workspace(8, 2, 128, 8, 1, ctypes.byref(n)) == OK and n.value > 0
    a = abg._TreeAttnArgs(**ATTN)
    assert lib.abg_tree_attn(ctypes.byref(a), WS, n.value - 1, None) == ESHAPE
    assert lib.abg_tree_attn(ctypes.byref(a), None, n.value, None) == EINVAL
    assert lib.abg_tree_attn(ctypes.byref(a), WS + 8, n.value, None) == EALIGN
    assert lib.abg_tree_attn(None, WS, n.value, None) == EINVAL
    assert lib.abg_tree_attn_workspace(8, 2, 128, 8, 1, None) == EINVAL
    assert lib.abg_tree_attn_workspace(8, 3, 128, 8, 1, ctypes.byref(n)) == ESHAPE
    assert lib.abg_tree_attn_workspace(8, 2, 128, 257, 1, ctypes.byref(n)) == ESHAPE


ACC = dict(logits=A, ld=1000, tok=A + STEP, parent=A + 2 * STEP, cu=A + 3 * STEP, best=A + 4 * STEP, rows=A + 5 * STEP,
           add=A + 6 * STEP, last=A + 7 * STEP, B=3, N=20, V=999, ws=WS, ws_bytes=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), ESHAPE), (dict(N=-1), ESHAPE), (dict(V=0), ESHAPE), (dict(ld=998), ESHAPE), (dict(ws_bytes=1), ESHAPE),
    *[({k: None}, EINVAL) for k in ("logits", "tok", "parent", "cu", "best", "rows", "add", "last", "ws")],
    (dict(logits=A + 2), EALIGN), (dict(ws=WS + 4), EALIGN), (dict(best=A + 4 * (19 * 1000 + 998)), EALIAS),
    (dict(rows=A + 4 * STEP + 76), EALIAS), (dict(add=A + 3 * STEP), EALIAS)])
def test_tree_accept_refuses(lib, change, status):
    assert lib.abg_tree_accept(*{**ACC, **change}.values(), None) == status


def test_plain_tree_plan_masks_are_ancestors():
    """The plain form itself, on a tree written out by hand."""
    mask, pos = ref.tree_plan(np.array([-1, 0, 0, 1, 3, -2, 5]), np.array([10]), np.array([0, 7]), 1)
    assert mask[:, 0].tolist() == [1, 3, 5, 11, 27, 0, 64]
    assert pos.tolist() == [10, 11, 11, 12, 13, 0, 10]


def test_plain_tree_attn_is_softmax_attention():
    """The plain form against a masked softmax over a dense matrix."""
    rng = np.random.default_rng(0)
    N, Hq, Hkv, D, page, n = 5, 4, 2, 64, 3, 10
    Kc, Vc = (rng.standard_normal((6, Hkv, page, D)) for _ in range(2))
    Kd, Vd = (rng.standard_normal((Hkv, N, D)) for _ in range(2))
    q, table = rng.standard_normal((N, Hq, D)), np.array([[4, 0, 5, 2]])
    bits = np.tri(N, 64, dtype=bool)
    y, _ = ref.tree_attn(q, Kc, Vc, table, [n], [0, N], Kd, Vd, bits)
    for hq in range(Hq):
        h = hq // 2
        K = np.concatenate([Kc[table[0], h].reshape(-1, D)[:n], Kd[h]])
        V = np.concatenate([Vc[table[0], h].reshape(-1, D)[:n], Vd[h]])
        s = q[:, hq] @ K.T / 8.0
        s[:, n:][~bits[:, :N]] = -np.inf
        p = np.exp(s - s.max(1, keepdims=True))
        assert np.allclose(y[:, hq], p / p.sum(1, keepdims=True) @ V, rtol=1e-12, atol=1e-13)


def bad_calls():
    """(call, words of the ValueError) with tensors that the binding refuses; all
    of them are on the CPU, which is the last thing each check looks at."""
    import torch
    i32, i64, f32, u8 = torch.int32, torch.int64, torch.float32, torch.uint8

    def z(*shape, dtype=i32):
        return torch.zeros(shape, dtype=dtype)

    def plan(**kw):
        a = dict(lens=z(2), add=z(2), cu=z(3), held=z(2), ends=z(2, dtype=i64), ring=z(9), table=z(2, 4), page=16,
                 slots=z(5, dtype=i64), pos=z(5), lens_out=z(2), held_out=z(2), ends_out=z(2, dtype=i64), info=z(2))
        return lambda: abg.page_plan(**{**a, **kw})

    def put(**kw):
        a = dict(k=z(3, 2, 64, dtype=f32), v=z(3, 2, 64, dtype=f32), Kc=z(1, 2, 8, 64, dtype=f32),
                 Vc=z(1, 2, 8, 64, dtype=f32))
        return lambda: abg.kv_put(**{**a, **kw})

    def attn(**kw):
        a = dict(q=z(3, 4, 64, dtype=f32), Kc=z(5, 2, 8, 64, dtype=f32), Vc=z(5, 2, 8, 64, dtype=f32), table=z(1, 4),
                 lens=z(1), cu=z(2), Kd=z(2, 3, 64, dtype=f32), Vd=z(2, 3, 64, dtype=f32), mask=z(3, 1, dtype=i64),
                 y=z(3, 4, 64, dtype=f32), ws=z(9, dtype=u8))
        return lambda: abg.tree_attn(**{**a, **kw})

    def accept(**kw):
        a = dict(logits=z(3, 9, dtype=f32), tok=z(3), parent=z(3), cu=z(2), best=z(3), rows=z(3), add=z(1), last=z(1),
                 ws=z(99, dtype=u8))
        return lambda: abg.tree_accept(**{**a, **kw})

    return [
        (plan(), "lens must be a contiguous torch.int32 CUDA tensor"), (plan(lens=3), "lens must be a tensor"),
        (lambda: abg.tree_plan(z(3), z(1), z(2), z(3, dtype=i64), z(3)), r"mask must be \[N\]\[words\]"),
        (lambda: abg.tree_plan(z(3), z(1), z(2), z(3, 1, dtype=i64), z(3)), "parent must be a contiguous"),
        (put(), "Kc must be a contiguous torch.float32 CUDA tensor"), (put(Vc=z(1, 2, 9, 64, dtype=f32)), "one shape"),
        (put(Kc=z(2, 8, 64, dtype=f32)), "one shape"),
        (put(Kc=z(1, 2, 8, 64), Vc=z(1, 2, 8, 64)), "Kc must be float32, bfloat16 or float16"),
        (attn(), "Kc must be a contiguous"), (attn(Kc=3), "Kc must be a tensor"),
        (accept(), "logits must be a float32 CUDA tensor"), (accept(logits=z(3, 9)), "logits must be a float32"),
        (accept(add=None), "add must be a tensor")]


def test_binding_refuses_wrong_tensors():
    for call, words in bad_calls():
        with pytest.raises(ValueError, match=words):
            call()


@pytest.mark.parametrize("given,words", [
    ("sin", "cos and sin must both be given"), ("cos", "cos and sin must both be given"),
    ("qo", "q and qo must both be given"), ("q", "q and qo must both be given")])
def test_binding_refuses_half_of_a_pair(given, words):
    """A rotation's sines without its cosines, or a place for q without q, is not
    taken for none of them."""
    import torch
    t = dict(sin=torch.zeros(5, 32), cos=torch.zeros(5, 32), q=torch.zeros(3, 4, 64), qo=torch.zeros(3, 4, 64))
    k = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match=words):
        abg.kv_put(k, k, torch.zeros(1, 2, 8, 64), torch.zeros(1, 2, 8, 64), pos=torch.zeros(3, dtype=torch.int32),
                   **{given: t[given]})
