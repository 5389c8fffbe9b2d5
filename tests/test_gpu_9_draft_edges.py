"""Where the draft-verification calls can go wrong: waits that give up, weights
far below the largest, rings and pages that run out."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from helpers import host
from test_gpu_9_draft import TYPES, U32, UNIT, attn_case, i32, i64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
abg = pytest.importorskip("affine_bit_group_gb300")


# ------------------------------------------------------ waits that give up ----
def attn_args(c):
    """The C call's arguments for tree_attn's of a 16-bit case."""
    ty = {torch.bfloat16: abg.SB_BF16, torch.float16: abg.SB_F16}[c["q"].dtype]
    N, Hq, D = c["q"].shape
    pages, Hkv, page, _ = c["Kc"].shape
    p = {k: c[k].data_ptr() for k in ("q", "Kc", "Vc", "table", "lens", "cu", "Kd", "Vd", "mask", "y")}
    return abg._TreeAttnArgs(**p, gate=c["gate"].data_ptr() if c["gate"] is not None else None, ysum=None,
                             B=len(c["lens"]), N=N, Hq=Hq, Hkv=Hkv, D=D, page=page, pages=pages,
                             width=c["table"].shape[1], drafts=c["Kd"].shape[1], words=c["mask"].shape[1],
                             max_span=c["max_span"], type=ty, y_type=ty)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,spans,item", [
    ([40000], [20], 0), ([40000], [64], 3), ([40000, 9000], [64, 30], 6),  # entries of units
    ([700] * 300, [2] * 300, 0), ([500] * 300, [5] * 300, 5)])             # entries of blocks
def test_tree_attn_ends_when_a_copy_never_comes(D, lens, spans, item):
    """The waits run out; the second launch has an entry for every unit all the
    same, so that it goes by nothing that the workspace held before; and the next
    call is right.  The workspace starts with entries of no rows (which are
    harmless) and a mark."""
    c, _ = attn_case(70, "bf16", 8, 2, D, 16, lens, spans, gate=False)
    n = abg.tree_attn_workspace(c["q"], c["Kc"], c["max_span"])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    abg.tree_attn(**c, ws=ws)
    want = c["y"].clone()
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    entries = ws[n - 24 * blocks:].view(torch.int32).view(blocks, 6)  # n0 h r0 rows first last, the last part of ws
    ws.zero_()
    entries[:, 0] = -77
    assert abg.device_status(clear=True) == 0
    a = attn_args(c)
    assert abg.library().abg_selftest_tree_attn_timeout(ctypes.byref(a), ws.data_ptr(), n, item,
                                                        torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    bits = abg.device_status(clear=True)
    assert bits == 1 | 256, bits  # waits of this kernel ran out; the waits for what was in flight did not
    rows = 256 if D < 256 else 128
    per = -(-64 * c["mask"].shape[1] * 4 // rows)  # entries a request and head
    e = host(entries)
    if len(lens) * 2 * per <= blocks:
        with_rows = [(b * 2 + h) * per + t for b, s in enumerate(spans) for h in range(2) for t in range(-(-4 * s // rows))]
        assert (e[with_rows, 0] != -77).all()
    else:
        assert (e[:, 0] != -77).all()
    written = e[(e[:, 0] != -77) & (e[:, 3] != 0)]
    assert (written[:, 4] >= 0).all() and (written[:, 4] < written[:, 5]).all() and (written[:, 5] < blocks).all()
    assert torch.equal(c["y"][sum(spans):], want[sum(spans):])
    abg.tree_attn(**c, ws=ws)
    assert torch.equal(c["y"], want) and abg.device_status(clear=True) == 0


def test_tree_attn_selftest_refuses_what_has_no_waits():
    c, _ = attn_case(71, "f16", 4, 2, 64, 16, [20], [3], gate=False)
    a, ws = attn_args(c), torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    call = abg.library().abg_selftest_tree_attn_timeout
    assert call(ctypes.byref(a), ws.data_ptr(), ws.numel(), -1, None) == 1
    a.type = a.y_type = abg.SB_F32
    assert call(ctypes.byref(a), ws.data_ptr(), ws.numel(), 0, None) == 1
    assert call(None, ws.data_ptr(), ws.numel(), 0, None) == 1


# ------------------------------------------------- weights far below the largest ----
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("tall", [
    [(0, 25.4)], [(0, 24.4)], [(70000, 20.7)], [(131071, 25.4)],
    [(0, 17.0), (90000, 24.7)], [(5, 25.4), (6, 18.0)]])  # token, log2 of its weight over the others'
def test_tree_attn_many_weights_far_below_the_largest(kind, D, tall):
    """131072 tokens of one score under one or two that are far above: the small
    weights together count, though each is below 2^-14 (f16's normal range) or
    2^-25 (half of its smallest) of the largest.  Requests that share the cache,
    so many that most of them are not cut (a piece has a largest score of its
    own); f32 result, one head, V = 1 where the score is small and 0 where it is
    large."""
    n, page, B, dtype = 131072, 128, 160, TYPES[kind]
    K, V = (np.zeros((n, D)) for _ in range(2))
    q = np.zeros(D)
    q[0], V[:] = 16.0, 1.0
    for t, lg in tall:
        K[t, 0], V[t] = lg * np.log(2) * np.sqrt(D) / q[0], 0.0
    K = torch.from_numpy(K).to(dtype)
    s = K.double().numpy()[:, 0] * q[0] / np.sqrt(D)
    w = np.exp(s - s.max())
    want = (w * V[:, 0]).sum() / w.sum()

    def pages(x):
        return torch.as_tensor(x).to(dtype).view(n // page, 1, page, D).cuda()

    y = torch.empty((B, 1, D), device="cuda")
    draft = torch.zeros((1, B, D), dtype=dtype, device="cuda")
    abg.tree_attn(torch.from_numpy(q).to(dtype).cuda().repeat(B, 1, 1), pages(K), pages(V),
                  i32(np.arange(n // page)[None].repeat(B, 0)), i32([n] * B), i32(np.arange(B + 1)), draft, draft,
                  i64(np.zeros((B, 1))), y)
    # the weights' rounding: half a unit in the last place of each, or 2^-32 of the
    # largest; in f32, of a sum of positive terms: a score's and a weight's few
    # roundings, sums of 16 at a time that may be cut off (two roundings each), joins
    bound = UNIT[kind] * 1.01 + n * 2.0**-32 + want * U32 * (2 * n / 16 + 600)
    assert np.abs(host(y) - want).max() <= bound, (host(y).min(), host(y).max(), want, bound)


# ------------------------------------------------------------- rings that are full ----
def test_page_plan_refuses_pages_that_the_ring_has_no_room_for():
    """Five entries, four of them free pages, and three requests that end: one page
    fits, the next request's do not, and neither does one after it.  The free pages
    stay what they are (a fourth request takes one of them in the same call)."""
    d = dict(lens=i32([5, 40, 7, 16]), add=i32([-1, -1, -1, 1]), cu=i32([0, 0, 0, 0, 1]), held=i32([1, 3, 1, 1]),
             ends=i64([2, 6]), ring=i32([90, 91, 92, 93, 94]), table=i32(np.arange(16).reshape(4, 4)))
    out = dict(slots=i64([7]), pos=i32([7]), lens_out=i32([9] * 4), held_out=i32([9] * 4), ends_out=i64([9, 9]),
               info=i32([9, 9]))
    for _ in range(2):
        abg.page_plan(**d, page=16, **out)
        assert host(out["lens_out"]).tolist() == [0, 40, 7, 17] and host(out["held_out"]).tolist() == [0, 3, 1, 2]
        assert host(out["ends_out"]).tolist() == [3, 7] and host(out["info"]).tolist() == [1, 2]
        assert host(d["ring"]).tolist() == [90, 0, 92, 93, 94]
        assert host(d["table"]).ravel().tolist() == [*range(13), 92, 14, 15]
        assert host(out["slots"]).tolist() == [92 * 16] and host(out["pos"]).tolist() == [16]


def test_page_plan_many_requests_end_in_a_small_ring():
    """1500 requests of three pages end, and the ring has room for 1000 pages: the
    first 333 requests' pages, over three rounds of the scan."""
    B = 1500
    table = i32(np.arange(4 * B).reshape(B, 4))
    ring, ends = i32(np.full(1100, -5)), i64([50, 150])
    lens_out, held_out, ends_out, info = i32(np.zeros(B)), i32(np.zeros(B)), i64([0, 0]), i32([0, 0])
    abg.page_plan(i32(np.full(B, 40)), i32(np.full(B, -1)), i32(np.zeros(B + 1)), i32(np.full(B, 3)), ends, ring, table, 16,
                  i64(np.zeros(0)), i32(np.zeros(0)), lens_out, held_out, ends_out, info)
    n = 333
    assert host(ends_out).tolist() == [50, 150 + 3 * n] and host(info).tolist() == [0, B - n]
    assert host(lens_out).tolist() == [0] * n + [40] * (B - n) and host(held_out).tolist() == [0] * n + [3] * (B - n)
    want = np.full(1100, -5)
    want[(150 + np.arange(3 * n)) % 1100] = (4 * np.arange(n)[:, None] + np.arange(3)).ravel()
    assert host(ring).tolist() == want.tolist()


# ------------------------------------------------------------- other streams ----
@pytest.mark.parametrize("handle", [False, True])
def test_default_workspace_belongs_to_the_call_s_stream(monkeypatch, handle):
    """A call on another stream without ws: the memory that it takes is not handed
    out to the current stream while the call may run."""
    c, _ = attn_case(81, "bf16", 8, 2, 128, 16, [900, 40], [9, 30], tail=0)
    abg.tree_attn(**c)
    want = c["y"].clone()
    x = torch.randn((39, 5000), device="cuda")
    tok, parent, cu = i32(np.zeros(39)), i32(np.full(39, -1)), c["cu"]
    out = [i32(np.zeros(39)), i32(np.zeros(39)), i32([0, 0]), i32([0, 0])]
    side, taken, plain = torch.cuda.Stream(), [], abg._bytes

    def spied(*a):
        t = plain(*a)
        taken.append((t.data_ptr(), t.numel()))
        return t

    monkeypatch.setattr(abg, "_bytes", spied)
    c["y"].zero_()
    torch.cuda.synchronize()
    stream = side.cuda_stream if handle else side
    abg.tree_attn(**c, stream=stream)
    abg.tree_accept(x, tok, parent, cu, *out, stream=stream)
    assert len(taken) == 2
    mine = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in taken for _ in range(8)]
    for p, n in taken:
        assert all(m.data_ptr() + m.numel() <= p or p + n <= m.data_ptr() for m in mine)
    side.synchronize()
    assert torch.equal(c["y"], want) and torch.equal(out[0], x.argmax(1).int())


# ------------------------------------------------------------ other threads ----
SLOW = """
#include <unistd.h>
#define SLOW(name) int name() { usleep(300000); return 0; }
SLOW(abg_page_plan) SLOW(abg_tree_plan) SLOW(abg_kv_put) SLOW(abg_tree_attn) SLOW(abg_tree_accept)
"""
TICKS = """
import ctypes, sys, threading, time
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # its calls take the place of the library's
import torch
sys.path[:0] = sys.argv[2:]
import test_gpu_9_draft as t
c, _ = t.attn_case(80, 'bf16', 4, 2, 64, 16, [20], [3], tail=0)
z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device='cuda')
ws = z(99, dtype=torch.uint8)
calls = dict(
    page_plan=lambda: t.abg.page_plan(z(2), z(2), z(3), z(2), z(2, dtype=torch.int64), z(9), z(2, 4), 16,
                                      z(5, dtype=torch.int64), z(5), z(2), z(2), z(2, dtype=torch.int64), z(2)),
    tree_plan=lambda: t.abg.tree_plan(z(3), z(1), z(2), z(3, 1, dtype=torch.int64), z(3)),
    kv_put=lambda: t.abg.kv_put(z(3, 2, 64, dtype=torch.float32), z(3, 2, 64, dtype=torch.float32),
                                z(1, 2, 8, 64, dtype=torch.float32), z(1, 2, 8, 64, dtype=torch.float32)),
    tree_attn=lambda: t.abg.tree_attn(**c, ws=ws),
    tree_accept=lambda: t.abg.tree_accept(z(3, 9, dtype=torch.float32), z(3), z(3), z(2), z(3), z(3), z(1), z(1), ws=ws))
ticks, done = [], False
def run():
    while not done:
        ticks.append(time.perf_counter())
        time.sleep(0.005)
thread = threading.Thread(target=run)
thread.start()
for name, call in calls.items():
    t0 = time.perf_counter()
    call()
    t1 = time.perf_counter()
    print(name, t1 - t0, sum(t0 + 0.1 < x < t0 + 0.25 for x in ticks))
done = True
thread.join()
"""


def test_calls_let_other_threads_run(tmp_path):
    """Calls that take long (as launches do when the queue is full) do not stop the
    other Python threads: the library's calls are replaced by ones that sleep."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    (tmp_path / "slow.c").write_text(SLOW)
    (tmp_path / "ticks.py").write_text(TICKS)
    lib = tmp_path / "slow.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(tmp_path / "slow.c")], check=True)
    out = subprocess.run([sys.executable, str(tmp_path / "ticks.py"), str(lib), os.path.dirname(here), here], check=True,
                         timeout=120, capture_output=True, text=True).stdout.split("\n")
    got = {name: (float(took), int(ticks)) for name, took, ticks in (line.split() for line in out if line)}
    assert len(got) == 5
    for name, (took, ticks) in got.items():
        assert took > 0.25 and ticks >= 3, (name, took, ticks)


# ------------------------------------------------------------- shapes of kv_put's tensors ----
def test_kv_put_refuses_rotations_of_another_width():
    """A rotation table with the head's whole width (each cosine twice) is not read
    as one with half of it and twice the positions."""
    k, pos = torch.ones((3, 1, 64), device="cuda"), i32([0, 1, 2])
    Kc, Vc = (torch.zeros((1, 1, 3, 64), device="cuda") for _ in range(2))
    t = {w: torch.ones((9, w), device="cuda") for w in (16, 32, 64)}
    for cos, sin in ((64, 64), (64, 32), (32, 64), (16, 16)):
        with pytest.raises(ValueError, match=r"cos and sin must be \[positions\]\[32\]"):
            abg.kv_put(k, k, Kc, Vc, cos=t[cos], sin=t[sin], pos=pos)
    assert not Kc.any() and not Vc.any()
    abg.kv_put(k, k, Kc, Vc, cos=t[32], sin=torch.zeros_like(t[32]), pos=pos)
    assert torch.equal(Kc, torch.ones_like(Kc))


def test_kv_put_takes_one_row_or_head_of_any_stride():
    """The strides of a single row and of a single head are never stepped over: a
    view whose are no multiple of 16 bytes is as good as another."""
    src = torch.randn(400, device="cuda")
    k = torch.as_strided(src, (1, 2, 64), (7, 64, 1))
    v = torch.as_strided(src, (1, 2, 64), (3, 128, 1), 16)
    Kc, Vc = (torch.zeros((1, 2, 4, 64), device="cuda") for _ in range(2))
    abg.kv_put(k, v, Kc, Vc)
    assert torch.equal(Kc[0, :, 0], k[0]) and torch.equal(Vc[0, :, 0], v[0])
    k = torch.as_strided(src, (3, 1, 64), (64, 5, 1))
    Kc, Vc = (torch.zeros((1, 1, 4, 64), device="cuda") for _ in range(2))
    abg.kv_put(k, k, Kc, Vc)
    assert torch.equal(Kc[0, 0, :3], k[:, 0]) and torch.equal(Vc[0, 0, :3], k[:, 0])


def test_kv_put_takes_flat_rotation_tables():
    k, pos = torch.randn((3, 1, 64), device="cuda"), i32([0, 2, 1])
    ang = torch.rand((3, 32), device="cuda")
    want, got = ([torch.zeros((1, 1, 3, 64), device="cuda") for _ in range(2)] for _ in range(2))
    abg.kv_put(k, k, *want, cos=ang.cos(), sin=ang.sin(), pos=pos)
    abg.kv_put(k, k, *got, cos=ang.cos(), sin=ang.sin().flatten(), pos=pos)
    assert torch.equal(got[0], want[0])
    abg.kv_put(k, k, *got, cos=ang.cos().flatten(), sin=ang.sin().unsqueeze(1), pos=pos)
    assert torch.equal(got[0], want[0])
    with pytest.raises(ValueError, match="cos and sin must be"):
        abg.kv_put(k, k, *got, cos=ang.cos().flatten()[:95], sin=ang.sin(), pos=pos)
