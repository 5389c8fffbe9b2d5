"""Refusals of the quantised cache's calls, without a GPU: every argument error
that the host can see has its documented status before any device work."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

import affine_bit_group_gb300 as abg
import kvq_ref as ref

OK, EINVAL, EALIGN, ESHAPE, EALIAS = 0, 1, 2, 3, 4
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x7F0000000000  # fake device addresses, 16 MB apart
STEP = 1 << 24


@pytest.fixture(scope="module")
def lib():
    return abg.library()


@pytest.mark.parametrize("ctype,cname", [(abg._KvqCache, "abg_kvq_cache"), (abg._KvqPutArgs, "abg_kvq_put_args"),
                                         (abg._KvqGetArgs, "abg_kvq_get_args"), (abg._KvqAttnArgs, "abg_kvq_attn_args")])
def test_struct_layout_matches_c(tmp_path, ctype, cname):
    fields = [f for f, _ in ctype._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text("\n".join(["#include <stdio.h>", "#include <stddef.h>", '#include "abg.h"', "int main(void){",
                               f'printf("%zu\\n", sizeof({cname}));'] +
                              [f'printf("%zu\\n", offsetof({cname}, {f}));' for f in fields] + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    out = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert out == [ctypes.sizeof(ctype)] + [getattr(ctype, f).offset for f in fields]


CACHE = dict(Kc=A, Ks=A + STEP, Vc=A + 2 * STEP, Vs=A + 3 * STEP, pages=8, Hkv=2, page=16, D=128, bits=4, group=64)


def call(lib, name, ctype, base, change, *more):
    args = {**base, **{k: v for k, v in change.items() if k not in CACHE}}
    c = abg._KvqCache(**{**CACHE, **{k: v for k, v in change.items() if k in CACHE}})
    return getattr(lib, name)(ctypes.byref(ctype(c=c, **args)), *more)


BAD_CACHE = [(dict(bits=3), EINVAL), (dict(bits=16), EINVAL), (dict(group=128), EINVAL), (dict(group=0), EINVAL),
             (dict(D=96), ESHAPE), (dict(D=32), ESHAPE), (dict(Hkv=0), ESHAPE), (dict(Hkv=65537), ESHAPE),
             (dict(page=0), ESHAPE), (dict(pages=-1), ESHAPE), (dict(pages=2**31), ESHAPE),
             (dict(pages=2**31 - 1, page=2**31 - 1), ESHAPE), (dict(pages=2**30, Hkv=4), ESHAPE),
             (dict(Kc=A + 8), EALIGN), (dict(Ks=A + STEP + 4), EALIGN), (dict(Vc=A + 2 * STEP + 4), EALIGN),
             (dict(Vs=A + 3 * STEP + 2), EALIGN), (dict(Kc=None), EINVAL), (dict(Vs=None), EINVAL)]

PUT = dict(q=A + 4 * STEP, k=A + 5 * STEP, v=A + 6 * STEP, q_row=512, q_head=128, k_row=256, k_head=128, v_row=256,
           v_head=128, rows=None, slots=A + 7 * STEP, qn_w=A + 8 * STEP, kn_w=A + 9 * STEP, cos=A + 10 * STEP,
           sin=A + 11 * STEP, pos=A + 12 * STEP, qo=A + 13 * STEP, N=10, src_rows=10, Hq=4, cos_rows=100, eps=1e-6,
           src_type=0, q_type=1)


@pytest.mark.parametrize("change,status", BAD_CACHE + [
    (dict(src_type=3), EINVAL), (dict(src_type=-1), EINVAL), (dict(q_type=3), EINVAL), (dict(src_type=2), EINVAL),
    (dict(Hq=0), ESHAPE), (dict(N=11), ESHAPE), (dict(N=-1), ESHAPE), (dict(src_rows=-1), ESHAPE), (dict(k_row=-256), ESHAPE),
    (dict(cos_rows=0), ESHAPE), (dict(N=0), OK), (dict(sin=None), EINVAL), (dict(qo=None), EINVAL), (dict(q=None), EINVAL),
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(pos=None), EINVAL), (dict(k=A + 5 * STEP + 4), EALIGN),
    (dict(k_row=257), EALIGN), (dict(v_head=130), EALIGN), (dict(q_row=513), EALIGN), (dict(slots=A + 7 * STEP + 4), EALIGN),
    (dict(pos=A + 12 * STEP + 1), EALIGN), (dict(qo=A + 5 * STEP), EALIAS), (dict(k=A + 64), EALIAS),
    (dict(Vs=A + STEP), EALIAS), (dict(Ks=A + 16 * 8 * 2 * 64 - 16), EALIAS), (dict(slots=A + 3 * STEP + 16), EALIAS),
    (dict(Vc=A + 13 * STEP + 10 * 4 * 128 * 2 - 16), EALIAS)])
def test_kvq_put_refuses(lib, change, status):
    assert call(lib, "abg_kvq_put", abg._KvqPutArgs, PUT, change, None) == status


GET = dict(slots=A + 4 * STEP, k=A + 5 * STEP, v=A + 6 * STEP, k_row=256, k_head=128, v_row=256, v_head=128, N=10, type=1)


@pytest.mark.parametrize("change,status", BAD_CACHE + [
    (dict(type=3), EINVAL), (dict(N=-1), ESHAPE), (dict(N=2**31), ESHAPE), (dict(N=0), OK), (dict(k_row=-8), ESHAPE),
    (dict(v_head=-8), ESHAPE), (dict(k=None, v=None), EINVAL), (dict(k=A + 5 * STEP + 8), EALIGN), (dict(k_row=260), EALIGN),
    (dict(v_head=132), EALIGN), (dict(slots=A + 4 * STEP + 4), EALIGN), (dict(k_row=248), EALIAS), (dict(k_head=64), EALIAS),
    (dict(v_row=0), EALIAS), (dict(v=A + 5 * STEP), EALIAS), (dict(v=A + 5 * STEP + 512), EALIAS),
    (dict(k=A + 2 * STEP), EALIAS), (dict(v=A + 3 * STEP), EALIAS), (dict(k=A + 4 * STEP), EALIAS),
    # interleaved rows of one buffer that meet: 2 heads of 128 in rows of 512, 192 columns apart; other row strides
    (dict(k_row=512, v_row=512, v=A + 5 * STEP + 384), EALIAS), (dict(k_row=512, v_row=1024, v=A + 5 * STEP + 512), EALIAS),
    (dict(k_row=512, v_row=512, v=A + 5 * STEP + 1024 + 640), EALIAS)])
def test_kvq_get_refuses(lib, change, status):
    assert call(lib, "abg_kvq_get", abg._KvqGetArgs, GET, change, None) == status


def test_kvq_get_rows_of_one_buffer_are_refused_where_they_meet_and_only_there(tmp_path):
    """The check's rule against every column written out: all places of v's rows
    beside k's, at equal strides exactly; at others never accepted where they meet."""
    prog = tmp_path / "rows.cpp"
    prog.write_text(r"""
#include "checks.cuh"
#include <cstdio>
#include <vector>
using namespace abg;
static bool meet(int64_t off, RowStrides a, RowStrides b, int64_t N, int64_t H, int64_t D) {
    std::vector<char> at(4096, 0);
    for (int64_t n = 0; n < N; ++n)
        for (int64_t h = 0; h < H; ++h)
            for (int64_t d = 0; d < D; ++d) at[n * a.row + h * a.head + d] = 1;
    for (int64_t n = 0; n < N; ++n)
        for (int64_t h = 0; h < H; ++h)
            for (int64_t d = 0; d < D; ++d)
                if (off + n * b.row + h * b.head + d < 4096 && at[off + n * b.row + h * b.head + d]) return true;
    return false;
}
int main() {
    const int64_t D = 2;
    long wrong = 0, apart = 0, met = 0, mixed = 0;
    for (int64_t N = 1; N <= 4; ++N)
        for (int64_t H = 1; H <= 4; ++H)
            for (int64_t row = 0; row <= 26; ++row)
                for (int64_t head = 0; head <= 26; ++head) {
                    const RowStrides a{row, head};
                    if (!rows_apart(a, N, H, D)) continue;
                    for (int64_t off = 0; off < (N - 1) * row + (H - 1) * head + D; ++off) {
                        // a single row's or head's stride is any number
                        const RowStrides b{N == 1 ? 7 : row, H == 1 ? 5 : head};
                        const bool m = meet(off, a, b, N, H, D);
                        wrong += rows_between(off, a, b, N, H, D) == m;
                        ++(m ? met : apart);
                        for (int64_t other = 0; other <= 12; other += 3)
                            for (const RowStrides &c : {RowStrides{row, other}, RowStrides{other, head}, RowStrides{other, other}})
                                if (rows_apart(c, N, H, D) && rows_between(off, a, c, N, H, D)) {
                                    wrong += meet(off, a, c, N, H, D);
                                    ++mixed;
                                }
                    }
                }
    std::printf("%ld %d %d %d\n", wrong, apart > 1000, met > 1000, mixed > 1000);
}
""")
    exe = tmp_path / "rows"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "affine_bit_group_gb300", "csrc"), "-I",
                    "/usr/local/cuda/include", str(prog), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out.split() == ["0", "1", "1", "1"]


ATTN = dict(q=A + 4 * STEP, table=A + 5 * STEP, lens=A + 6 * STEP, cu=A + 7 * STEP, Kd=A + 8 * STEP, Vd=A + 9 * STEP,
            mask=A + 10 * STEP, gate=A + 11 * STEP, y=A + 12 * STEP, ysum=A + 13 * STEP, B=3, N=20, Hq=8, width=4, drafts=20,
            words=1, max_span=9, type=1, y_type=0)
WS = A + 16 * STEP


@pytest.mark.parametrize("change,status", BAD_CACHE + [
    (dict(type=3), EINVAL), (dict(y_type=2), EINVAL), (dict(type=2, y_type=1), EINVAL), (dict(y_type=1), EINVAL),
    (dict(Hq=7), ESHAPE), (dict(Hq=0), ESHAPE), (dict(Hq=1), ESHAPE), (dict(B=0), ESHAPE), (dict(N=-1), ESHAPE),
    (dict(N=21), ESHAPE), (dict(words=0), ESHAPE), (dict(words=5), ESHAPE), (dict(max_span=0), ESHAPE),
    (dict(max_span=65), ESHAPE), (dict(width=-1), ESHAPE), (dict(width=2**27, page=16), ESHAPE), (dict(N=0), OK),
    *[({k: None}, EINVAL) for k in ("q", "table", "lens", "cu", "Kd", "Vd", "mask", "y")],
    (dict(q=A + 4 * STEP + 8), EALIGN), (dict(gate=A + 11 * STEP + 4), EALIGN), (dict(mask=A + 10 * STEP + 4), EALIGN),
    (dict(table=A + 5 * STEP + 2), EALIGN), (dict(ysum=A + 13 * STEP + 2), EALIGN), (dict(y=A + 4 * STEP), EALIAS),
    (dict(y=A), EALIAS), (dict(y=A + 3 * STEP), EALIAS), (dict(ysum=A + 12 * STEP + 16), EALIAS), (dict(y=WS + 1024), EALIAS),
    (dict(Vd=WS), EALIAS), (dict(N=0, width=2**27 - 64, page=16), ESHAPE), (dict(N=0, width=2**27 - 128, page=16), OK)])
def test_kvq_attn_refuses(lib, change, status):
    assert call(lib, "abg_kvq_attn", abg._KvqAttnArgs, ATTN, change, WS, 1 << 40, None) == status


def test_kvq_attn_refuses_a_small_or_no_workspace(lib):
    n = ctypes.c_int64()
    c = abg._KvqCache(**CACHE)
    assert lib.abg_kvq_attn_workspace(ctypes.byref(c), 8, 9, 1, ctypes.byref(n)) == OK and n.value > 0
    assert call(lib, "abg_kvq_attn", abg._KvqAttnArgs, ATTN, {}, WS, n.value - 1, None) == ESHAPE
    assert call(lib, "abg_kvq_attn", abg._KvqAttnArgs, ATTN, {}, None, n.value, None) == EINVAL
    assert call(lib, "abg_kvq_attn", abg._KvqAttnArgs, ATTN, {}, WS + 8, n.value, None) == EALIGN
    for change in (dict(bits=5), dict(group=48)):
        assert lib.abg_kvq_attn_workspace(ctypes.byref(abg._KvqCache(**{**CACHE, **change})), 8, 9, 1, ctypes.byref(n)) == EINVAL
    for Hq, span in ((7, 9), (8, 0), (8, 257)):
        assert lib.abg_kvq_attn_workspace(ctypes.byref(c), Hq, span, 1, ctypes.byref(n)) == ESHAPE
    assert lib.abg_kvq_attn_workspace(None, 8, 9, 1, ctypes.byref(n)) == EINVAL
    assert lib.abg_kvq_attn_workspace(ctypes.byref(c), 8, 9, 1, None) == EINVAL


def test_no_arguments_at_all(lib):
    assert lib.abg_kvq_put(None, None) == lib.abg_kvq_get(None, None) == lib.abg_kvq_attn(None, None, 0, None) == EINVAL


def test_binding_refuses_before_any_device_work():
    torch = pytest.importorskip("torch")
    k = torch.zeros((3, 2, 64))
    with pytest.raises(ValueError, match="bits must be"):
        abg.kvq_cache(1, 2, 3, 64, bits=5, device="cpu")
    cache = abg.kvq_cache(1, 2, 3, 64, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(1, 2, 3, 8), (1, 2, 3, 1, 2)] * 2
    with pytest.raises(ValueError, match="Kc must be a contiguous torch.int32 CUDA tensor"):
        abg.kvq_put(k, k, cache)
    with pytest.raises(ValueError, match="Kc must be a contiguous torch.int32 CUDA tensor"):
        abg.kvq_get(cache, k, k)
    with pytest.raises(ValueError, match="cos and sin"):
        abg.kvq_put(k, k, cache, cos=k)
    with pytest.raises(ValueError, match="k or v"):
        abg.kvq_get(cache, None, None)


# ------------------------------------------------------- the format's rule ----
def test_reference_rule_on_known_groups():
    """By hand: -3 .. 12 in steps of 1 has scale 1, bias -3 and codes 0 .. 15; one
    value far out; equal values; a NaN."""
    x = np.zeros((4, 32), np.float32)
    x[0] = np.tile(np.arange(16), 2) - 3.0
    x[1, 5] = 30.0
    x[2] = 0.1
    x[3, 7] = np.nan
    words, pairs = ref.quantise(x, 4, 32)
    assert pairs[0].tolist() == [[1.0, -3.0]] and ref.codes(words[0], 4).tolist() == [*range(16)] * 2
    assert pairs[1].tolist() == [[2.0, 0.0]] and ref.codes(words[1], 4).tolist() == [15 * (i == 5) for i in range(32)]
    assert pairs[2].tolist() == [[0.0, float(np.float16(0.1))]] and not words[2].any()
    assert pairs[3].view(np.uint16).tolist() == [[0x7FFF, 0x7FFF]] and not words[3].any()
    assert words[0, 0] == 0x76543210
