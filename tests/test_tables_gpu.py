"""The step tables on the GPU against the oracle, which takes one request after the other; whole numbers, so equal."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle.q4 import ref_build_tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
BITS = dict(bad_page=1, too_long=2, bad_chunk=8, no_pages=32)


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def state(B, P, stride, spare, seed, max_len, unused=5):
    """Lengths, a table of distinct pages and a stack of the spare ones (pool: all of them and some unused)."""
    r = np.random.default_rng(seed)
    lens = r.integers(0, max_len + 1, B)
    held = -(-lens // P)
    ids = r.permutation(int(held.sum()) + spare + unused)
    pt = r.integers(-9, 0, (B, stride))  # entries past a row's pages: anything
    at = 0
    for b in range(B):
        pt[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(len(ids), -7)
    free[:spare] = ids[at:at + spare]
    return lens, pt, free


def run(ops, lens, new, pt, free, count, P, max_tokens, in_place=False):
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    d = dict(lens=i32(lens), new=i32(new), pt=i32(pt), free=i32(free), count=i32([count]))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(kv_lens=d["lens"], free_left=d["count"]) if in_place else {}
    kv, cu, slots, left = ops.build_tables(d["lens"], d["new"], d["pt"], d["free"], d["count"], page_size=P,
                                           max_tokens=max_tokens, device_error=err, **kw)
    return dict(kv_lens=kv, cu=cu, slots=slots, table=d["pt"], free=d["free"], left=left), int(err)


def compare(got, err, want):
    for key in ("kv_lens", "cu", "slots", "table", "free"):
        assert np.array_equal(got[key].cpu().numpy(), want[key]), key
    assert int(got["left"]) == want["left"]
    assert err == sum(BITS[b] for b in want["bits"])


@pytest.mark.parametrize("B", [1, 2, 31, 33, 200, 1025, 2500, 8192])
@pytest.mark.parametrize("in_place", [False, True])
def test_random_steps(ops, B, in_place):
    P = [16, 48, 64, 256][B % 4]
    stride = 12
    r = np.random.default_rng(B)
    for seed, spare in ((0, 4 * B), (1, B // 2), (2, 0)):
        lens, pt, free = state(B, P, stride, spare, seed, max_len=10 * P)
        new = np.where(r.random(B) < 0.5, 1, r.integers(0, 3 * P, B))
        new[r.random(B) < 0.15] = -1
        total = int(np.maximum(new, 0).sum())
        for most in (total + 7, total, total // 2):
            want = ref_build_tables(lens, new, pt, free, spare, P, most)
            got, err = run(ops, lens, new, pt, free, spare, P, most, in_place)
            compare(got, err, want)


def test_pages_returned_are_taken_in_the_same_step(ops):
    # empty stack: the request before the ended one takes the pages it returns
    lens, pt = [0, 40], np.array([[-1, -1, -1], [4, 2, 9]])
    free = np.zeros(10, dtype=np.int64)
    want = ref_build_tables(lens, [33, -1], pt, free, 0, 16, 40)
    assert list(want["table"][0]) == [9, 2, 4] and not want["bits"]
    compare(*run(ops, lens, [33, -1], pt, free, 0, 16, 40), want)


def test_refused_requests_keep_their_state_and_can_ask_again(ops):
    lens, pt = [16, 16, 5], np.array([[0, -1], [1, -1], [2, -1]])
    free = np.array([7, 0, 0, 0, 0, 0, 0, 0])
    got, err = run(ops, lens, [1, 1, 1], pt, free, 1, 16, 3)
    assert err == 32
    assert got["kv_lens"].tolist() == [17, 16, 6] and got["slots"].tolist() == [7 * 16, -1, 2 * 16 + 5]
    assert got["cu"].tolist() == [0, 1, 2, 3] and got["table"][1].tolist() == [1, -1] and int(got["left"]) == 0


def test_row_that_cannot_hold_a_request(ops):
    lens, pt = [30, 10], np.array([[0, 1], [2, -1]])
    free = np.array([5, 6, 0, 0, 0, 0, 0, 0])
    for n in (3, 2 ** 31 - 1):
        got, err = run(ops, lens, [n, 7], pt, free, 2, 16, 20)
        assert err & 2 and got["kv_lens"].tolist() == [30, 17]
        assert got["slots"][:3].tolist() == [-1, -1, -1] and int(got["left"]) == 1
    # packed offsets past 2^31 - 1 are held there, and nothing gets a slot outside its request
    got, err = run(ops, [0, 0, 0], [2 ** 31 - 1, 2 ** 31 - 1, 4], np.zeros((3, 2)), free, 2, 16, 20)
    assert err & 2 and (got["slots"] < 0).all() and got["cu"].tolist() == [0] + [2 ** 31 - 1] * 3


def test_bad_lengths_and_page_ids(ops):
    pt = np.array([[0, 1], [2, -1]])
    free = np.array([99, -3, 3, 4])
    got, err = run(ops, [-5, 16], [1, 1], pt, free, 2, 16, 2)   # a negative length; a bad id on the stack
    assert err == 2 | 1 and got["slots"].tolist() == [-1, -1] and got["kv_lens"].tolist() == [-5, 17]
    got, err = run(ops, [32, 16], [-1, -1], pt, free, 3, 16, 2)  # more pages than the pool has come back
    assert err == 1 and int(got["left"]) == 4 and got["free"].tolist() == [99, -3, 3, 0]


def test_no_tokens_and_no_requests(ops):
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    kv, cu, slots, left = ops.build_tables(z(2), z(2), z(2, 3), z(4), z(1), page_size=16, max_tokens=0)
    assert kv.tolist() == [0, 0] and cu.tolist() == [0, 0, 0] and slots.shape == (0,)


def test_repeats_give_the_same(ops):
    lens, pt, free = state(300, 64, 20, 400, 4, 1000)
    new = np.ones(300, dtype=np.int64)
    new[::17] = -1
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    d = [i32(x) for x in (lens, new, pt, free, [400])]
    want = ref_build_tables(lens, new, pt, free, 400, 64, 300)
    for _ in range(4):
        kv, cu, slots, left = ops.build_tables(*d, page_size=64, max_tokens=300)
        assert np.array_equal(slots.cpu().numpy(), want["slots"]) and int(left) == want["left"]
        assert np.array_equal(d[2].cpu().numpy(), want["table"]) and np.array_equal(kv.cpu().numpy(), want["kv_lens"])
