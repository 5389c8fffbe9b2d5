"""Draft decoding end to end: a small synthetic decoder with attention, its
caches in pages, and trees of drafts, against the same decoder one token at a
time."""
from __future__ import annotations

import numpy as np
import pytest

from affine_bit_group_gb300 import synth
from helpers import host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
abg = pytest.importorskip("affine_bit_group_gb300")
from affine_bit_group_gb300 import decode, draft  # noqa: E402

V, HIDDEN, D = 1500, 512, 64


@pytest.fixture(scope="module")
def weights():
    model, _ = synth.decode_model(seed=31, n_layers=2, hidden=HIDDEN, mlp=1024, head_rows=V, q_rows=8 * D, kv_rows=2 * D)
    embed = np.random.default_rng(32).standard_normal((V, HIDDEN)).astype(np.float32)
    return decode.DeviceModel.upload(model), torch.from_numpy(embed).cuda()


def i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


def decoder(weights, requests, cache=torch.float32, pages=64):
    return draft.DraftDecoder(*weights, D=D, requests=requests, pages=pages, page=4, max_len=200, rows=40, cache=cache)


def one_by_one(weights, first, count, cache):
    """count tokens after each of `first`, a single draft a step."""
    B = len(first)
    dec, tok, out = decoder(weights, B, cache), i32(first), []
    for _ in range(count):
        _, add, last = dec.step(tok, i32([-1] * B), i32(np.arange(B + 1)), 1)
        assert host(add).tolist() == [1] * B
        tok = last.clone()
        out.append(host(tok))
    return np.stack(out, 1), dec


@pytest.mark.parametrize("cache", [torch.float32, torch.bfloat16, torch.float16])
def test_drafts_give_the_tokens_of_one_by_one(weights, cache):
    """Trees whose one branch is the right continuation: each step accepts it
    whole, and the tokens and the cached lengths are those of single steps."""
    rng = np.random.default_rng(33)
    first = [7, 1200, 44]
    want, _ = one_by_one(weights, first, 24, cache)
    dec = decoder(weights, 3, cache)
    at = np.zeros(3, int)   # tokens known after the first
    got = [[] for _ in first]
    for step in range(6):
        depth = [3, 1, 2] if step % 2 else [0, 4, 1]  # right guesses of each request
        tok, parent, cu = [], [], [0]
        for b, d in enumerate(depth):
            known = first[b] if at[b] == 0 else want[b, at[b] - 1]
            t, p = [known], [-1]
            for i in range(d):
                t.append(rng.integers(0, V)), p.append(len(t) - 2 if i == 0 else right)  # a wrong sibling first
                t.append(want[b, at[b] + i]), p.append(p[-1])
                right = len(t) - 1
            tok, parent = tok + t, parent + p
            cu.append(len(tok))
        rows, add, last = dec.step(i32(tok), i32(parent), i32(cu), max(np.diff(cu)))
        assert host(add).tolist() == [d + 1 for d in depth]
        rows = host(rows)
        for b, d in enumerate(depth):
            path = [tok[r] for r in rows[cu[b]:cu[b] + d + 1]]
            got[b] += path[1:] + [int(last[b])]
            at[b] += d + 1
            assert got[b] == want[b, :at[b]].tolist()
    assert host(dec.lens[0]).tolist() == at.tolist()
    assert host(dec.held[0]).tolist() == (-(-at // 4)).tolist()
    assert abg.device_status(clear=True) == 0


def test_wrong_drafts_cost_nothing_and_ended_requests_give_their_pages_back(weights):
    want, _ = one_by_one(weights, [3, 9], 6, torch.float32)
    dec = decoder(weights, 2, pages=5)
    tok = [3, 9]
    for i in range(6):  # three wrong drafts beside each token
        t, p, cu = [], [], [0]
        for b in range(2):
            t += [tok[b]] + [(want[b, i] + 1 + k) % V for k in range(3)]
            p += [-1, 0, 0, 1]
            cu.append(len(t))
        _, add, last = dec.step(i32(t), i32(p), i32(cu), 4)
        assert host(add).tolist() == [1, 1] and host(dec.info).tolist()[1] == 0
        tok = host(last).tolist()
        assert tok == want[:, i].tolist()
    assert host(dec.held[0]).tolist() == [2, 2]
    dec.release(torch.tensor([True, False]))
    assert host(dec.held[0]).tolist() == [0, 2] and host(dec.lens[0]).tolist() == [0, 6]
    ends = host(dec.ends[0])
    assert ends[1] - ends[0] == 3
    # the freed pages serve the next tokens: a new request in row 0
    fresh, _ = one_by_one(weights, [500], 5, torch.float32)
    tok = [500, tok[1]]
    for i in range(5):
        _, add, last = dec.step(i32(tok), i32([-1, -1]), i32([0, 1, 2]), 1)
        assert host(dec.info).tolist()[1] == 0
        tok = host(last).tolist()
        assert tok[0] == fresh[0, i]


def test_a_step_that_runs_out_of_pages_says_so(weights):
    dec = decoder(weights, 2, pages=1)
    dec.step(i32([1, 2]), i32([-1, -1]), i32([0, 1, 2]), 1)
    assert host(dec.info).tolist() == [1, 1] and host(dec.lens[0]).tolist() == [1, 0]


def test_a_request_that_is_refused_keeps_its_token(weights):
    """Two requests and one page: the second is not accepted, its last token stays
    the next step's first, and what follows is what follows without the refusal."""
    want, _ = one_by_one(weights, [1, 2], 4, torch.float32)
    dec = decoder(weights, 2, pages=1)
    # request 1's second guess is right, but there is no page for either token
    rows, add, last = dec.step(i32([1, 2, 3, want[1, 0]]), i32([-1, -1, 0, 0]), i32([0, 1, 4]), 3)
    assert host(dec.info).tolist() == [1, 1] and host(dec.lens[0]).tolist() == [1, 0]
    assert host(add).tolist() == [1, 0] and host(rows).tolist() == [0, -1, -1, -1]
    assert host(last).tolist() == [want[0, 0], 2]
    dec.release(torch.tensor([True, False]))
    tok = last[1:].clone()
    for i in range(4):  # the page is request 1's now; request 0 has no drafts
        rows, add, last = dec.step(tok, i32([-1]), i32([0, 0, 1]), 1)
        assert host(dec.info).tolist()[1] == 0 and host(add).tolist() == [0, 1]
        assert host(last).tolist() == [-1, want[1, i]] and host(rows).tolist() == [0]
        tok = last[1:].clone()
    rows, add, last = dec.step(tok, i32([-1]), i32([0, 0, 1]), 1)  # a fifth token, and no second page
    assert host(add).tolist() == [0, 0] and host(last).tolist() == [-1, want[1, 3]] and host(rows).tolist() == [-1]


def test_the_last_page_is_used_to_its_end(weights):
    """max_len 10 in pages of 4: the table holds 12 tokens, and all of them have a
    rotation; a thirteenth is refused."""
    want, _ = one_by_one(weights, [7], 12, torch.float32)
    dec = draft.DraftDecoder(*weights, D=D, requests=1, pages=4, page=4, max_len=10, rows=40)
    tok = i32([7])
    for i in range(12):
        _, add, last = dec.step(tok, i32([-1]), i32([0, 1]), 1)
        assert host(add).tolist() == [1] and host(last).tolist() == [want[0, i]], i
        tok = last.clone()
    dec.step(tok, i32([-1]), i32([0, 1]), 1)
    assert host(dec.info).tolist() == [0, 1] and host(dec.lens[0]).tolist() == [12]
