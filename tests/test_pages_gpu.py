"""Forking, releasing, compacting and copying of pages on the GPU, against the oracle: whole numbers and bytes, so
everything has to be equal."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle.pages import pages_for, ref_compact, ref_fork, ref_release

pytestmark = pytest.mark.gpu
DEV = "cuda"
BITS = {"bad_page": 1, "too_long": 2, "bad_slot": 16, "no_pages": 32}


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def word(bits):
    return sum(BITS[b] for b in bits)


class State:
    """Requests with pages of their own in a shuffled pool; some pages are nobody's."""

    def __init__(self, lens, P, stride, spare, seed, nobody=3):
        rng = np.random.default_rng(seed)
        n = [pages_for(x, P) for x in lens]
        self.P = P
        self.n_pages = sum(n) + spare + nobody
        pages = rng.permutation(self.n_pages)
        self.table = rng.integers(0, self.n_pages, (len(lens), stride))  # what is behind a row's pages is no page of it
        at = 0
        for b, k in enumerate(n):
            self.table[b, :k] = pages[at:at + k]
            at += k
        self.free = rng.integers(0, self.n_pages, self.n_pages)
        self.free[:spare] = pages[at:at + spare]
        self.count = spare
        self.lens = np.array(lens)
        self.refs = np.zeros(self.n_pages, dtype=np.int64)

    def dev(self):
        return dict(lens=i32(self.lens), table=i32(self.table), refs=i32(self.refs), free=i32(self.free),
                    count=i32([self.count]))


def check_fork(ops, s, source, in_place=False):
    d, err = s.dev(), i32([0])
    want = ref_fork(source, s.lens, s.table, s.refs, s.free, s.count, s.P)
    kw = dict(kv_lens=d["lens"], free_left=d["count"]) if in_place else {}
    kv, src, dst, left = ops.fork_pages(i32(source), d["lens"], d["table"], d["refs"], d["free"], d["count"],
                                        page_size=s.P, device_error=err, **kw)
    for got, name in ((kv, "kv_lens"), (d["table"], "table"), (d["refs"], "refs"), (src, "src"), (dst, "dst")):
        assert np.array_equal(got.cpu().numpy(), want[name]), name
    assert int(left) == want["left"] and int(err) == word(want["bits"])
    assert torch.equal(d["free"], i32(s.free))
    if not in_place:
        assert torch.equal(d["lens"], i32(s.lens)) and int(d["count"]) == s.count
    s.lens, s.table, s.refs, s.count = want["kv_lens"], want["table"], want["refs"], want["left"]
    return want


def check_release(ops, s, new, in_place=False):
    d, err = s.dev(), i32([0])
    want = ref_release(s.lens, new, s.table, s.refs, s.free, s.count, s.P)
    kw = dict(kv_lens=d["lens"], free_left=d["count"]) if in_place else {}
    kv, left = ops.release_pages(d["lens"], i32(new), d["table"], d["refs"], d["free"], d["count"], page_size=s.P,
                                 device_error=err, **kw)
    for got, name in ((kv, "kv_lens"), (d["refs"], "refs"), (d["free"], "free")):
        assert np.array_equal(got.cpu().numpy(), want[name]), name
    assert int(left) == want["left"] and int(err) == word(want["bits"]) and torch.equal(d["table"], i32(s.table))
    s.lens, s.refs, s.free, s.count = want["kv_lens"], want["refs"], want["free"], want["left"]
    return want


def check_compact(ops, s, refs=True):
    d, err = s.dev(), i32([0])
    want = ref_compact(s.lens, s.table, s.refs, s.free, s.count, s.P)
    src, dst, moves = ops.compact_pages(d["lens"], d["table"], d["free"], d["count"], page_size=s.P,
                                        page_refs=d["refs"] if refs else None, device_error=err)
    for got, name in ((d["table"], "table"), (d["free"], "free"), (src, "src"), (dst, "dst")):
        assert np.array_equal(got.cpu().numpy(), want[name]), name
    assert np.array_equal(d["refs"].cpu().numpy(), want["refs"] if refs else s.refs)
    assert int(moves) == want["moves"] and int(err) == word(want["bits"])
    s.table, s.refs, s.free = want["table"], want["refs"], want["free"]
    return want


def whole(s):
    """Every known page is on the stack or has as many owners as its counter says."""
    owners = np.zeros(s.n_pages, dtype=int)
    for b, L in enumerate(s.lens):
        for c in range(pages_for(L, s.P)):
            owners[s.table[b, c]] += 1
    stack = list(s.free[:s.count])
    assert len(set(stack)) == len(stack) and not owners[stack].any()
    assert np.array_equal(s.refs, np.maximum(owners - 1, 0))


# ------------------------------------------------------------------ each call

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,P", [([40], 16), ([100, 64, 1, 0, 257], 64), ([16, 15, 17], 16), ([3000, 2048], 48)])
def test_fork(ops, lens, P, in_place):
    B = len(lens) + 6
    s = State(lens + [0] * 6, P, pages_for(max(lens), P) + 1, 9, 1)
    source = np.full(B, -1)
    source[-6:] = np.arange(6) % len(lens)
    check_fork(ops, s, source, in_place)
    whole(s)


def test_fork_refusals(ops):
    """Too few pages, rows that hold tokens, sources that are no rows, a source longer than its row, a fork of a fork,
    a row of itself: each reported, the row left."""
    s = State([40, 32, 0, 0, 0, 0, 0, 0, 0, 60], 16, 4, 2, 2)
    source = [1, -1, 0, 0, 0, 1, 10, 2, 8, -1]
    want = check_fork(ops, s, source)
    assert want["bits"] == {"no_pages", "bad_slot"} and list(want["kv_lens"][:9]) == [40, 32, 40, 40, 0, 32, 0, 0, 0]
    whole(s)
    s = State([16, 0], 16, 2, 1, 3)
    s.lens[0] = 33
    want = check_fork(ops, s, [-1, 0])
    assert want["bits"] == {"too_long"}


@pytest.mark.parametrize("in_place", [False, True])
def test_release(ops, in_place):
    s = State([100, 64, 1, 0, 257, 33, 0, 0, 0, 0], 16, 20, 12, 4)
    check_fork(ops, s, [-1, -1, -1, -1, -1, -1, 4, 4, 0, 4])
    check_release(ops, s, [1, -1, -1, -1, -1, 0, 1, -1, -1, 1], in_place)
    whole(s)
    check_release(ops, s, [-1] * 10, in_place)  # all end: every page comes back
    whole(s)
    assert not s.refs.any()


def test_release_reports_what_cannot_be(ops):
    """A page of two ended rows that it knows no second owner of comes back once; a full stack drops pages; page ids
    out of range are skipped."""
    s = State([32, 32], 16, 2, 0, 5)
    s.table[1, 0] = s.table[0, 0]
    want = check_release(ops, s, [-1, -1])
    assert want["bits"] == {"bad_page"} and want["left"] == 3
    s = State([32], 16, 2, 3, 6, nobody=0)
    s.count = s.n_pages - 1
    want = check_release(ops, s, [-1])
    assert want["bits"] == {"bad_page"} and want["left"] == s.n_pages
    s = State([48], 16, 3, 1, 7)
    d, err = s.dev(), i32([0])
    d["table"][0, 1] = -4
    d["table"][0, 2] = 1 << 30
    _, left = ops.release_pages(d["lens"], i32([-1]), d["table"], d["refs"], d["free"], d["count"], page_size=16,
                                device_error=err)
    assert int(err) == 1 and int(left) == 2 and int(d["free"][1]) == s.table[0, 0]


@pytest.mark.parametrize("seed", range(4))
def test_release_of_a_page_twice_in_a_row(ops, seed):
    """Entries next to each other, in the same 32 of a row, far apart, and in other rows: back once, no place left out."""
    rng = np.random.default_rng(seed)
    s = State([100 * 16, 40 * 16, 3 * 16, 17], 16, 101, 5, 30 + seed)
    at = [(0, 0), (0, 1), (0, 40), (1, 39), (2, 2)]
    page = s.table[0, 7]
    for b, c in at[:2 + seed]:
        s.table[b, c] = page
    for _ in range(seed):
        s.table[1, rng.integers(40)] = s.table[1, rng.integers(40)]
    want = check_release(ops, s, [-1, -1, -1, 2])
    assert want["bits"] == {"bad_page"} and not want["refs"].any()
    stack = want["free"][:want["left"]]
    assert len(set(stack.tolist())) == len(stack)


@pytest.mark.parametrize("seed", range(4))
def test_compact(ops, seed):
    rng = np.random.default_rng(seed)
    lens = list(rng.integers(0, 200, 7)) + [0] * 3
    s = State(lens, 16, 14, 10, seed + 10)
    check_fork(ops, s, [-1] * 7 + [0, 0, 3])
    check_release(ops, s, [1, -1, 1, -1, 1, 1, -1, 1, 1, -1])
    check_compact(ops, s)
    whole(s)
    check_compact(ops, s)  # nothing left to move
    stack = s.free[:s.count]
    assert np.all(np.diff(stack) < 0)


def test_compact_edges(ops):
    for lens, spare in (([0, 0], 5), ([40, 3], 0), ([0], 0), ([16] * 70, 33)):
        s = State(lens, 16, 4, spare, len(lens), nobody=2)
        check_compact(ops, s, refs=False)
        whole(s)
    s = State([40, 33], 16, 3, 4, 9)   # a live page on the stack stays in use
    s.free[1] = s.table[0, 1]
    d, err = s.dev(), i32([0])
    want = ref_compact(s.lens, s.table, s.refs, s.free, s.count, 16)
    src, dst, moves = ops.compact_pages(d["lens"], d["table"], d["free"], d["count"], page_size=16, device_error=err)
    assert int(err) == 1 and int(moves) == want["moves"] and np.array_equal(d["table"].cpu().numpy(), want["table"])


@pytest.mark.parametrize("lens,spoil", [([40, 33], "live"), ([40, 33], "twice"), ([16] * 70, "both")])
def test_compact_of_a_spoiled_stack(ops, lens, spoil):
    """A live page on the stack, a page on it twice: what is taken off the stack afterwards is no live page."""
    s = State(lens, 16, 4, 9, 21)
    if spoil in ("live", "both"):
        s.free[7] = s.table[0, 0]
    if spoil in ("twice", "both"):
        s.free[2] = s.free[5]
    want = check_compact(ops, s, refs=False)
    assert want["bits"] == {"bad_page"}
    live = {int(s.table[b, c]) for b, L in enumerate(lens) for c in range(pages_for(L, 16))}
    got = [int(x) for x in s.free[:s.count]]
    kept = [x for x in got if x >= 0]
    assert not live & set(kept) and len(set(kept)) == len(kept) and got[:len(got) - len(kept)] == [-1] * (len(got) - len(kept))


def test_compact_without_rows(ops):
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    free = i32([5, 1, 3, 0, 0, 0])
    src, dst, moves = ops.compact_pages(e, torch.empty((0, 4), dtype=torch.int32, device=DEV), free, i32([3]), page_size=16)
    assert int(moves) == 0 and free.tolist() == [5, 3, 1, 0, 0, 0] and bool((src == -1).all())


@pytest.mark.parametrize("B,P,mean,pages", [(8192, 16, 100, 0), (1000, 64, 900, 0), (300, 16, 700, 500000)])
def test_many_requests(ops, B, P, mean, pages):
    """As many requests as a call takes, and a pool near the largest that can be compacted."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 2 * mean, B)
    kids = rng.permutation(B)[:B // 3]
    lens[kids] = 0
    s = State(list(lens), P, pages_for(2 * mean, P), B, 20, nobody=pages)
    source = np.full(B, -1)
    source[kids] = rng.integers(0, B, len(kids))
    check_fork(ops, s, source)
    check_release(ops, s, np.where(rng.random(B) < 0.4, -1, 1))
    check_compact(ops, s)
    whole(s)


def test_no_requests(ops):
    e, refs = torch.empty(0, dtype=torch.int32, device=DEV), i32([0] * 4)
    table = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    *_, left = ops.fork_pages(e, e, table, refs, refs, i32([3]), page_size=16)
    assert int(left) == 3
    _, left = ops.release_pages(e, e, table, refs, refs, i32([2]), page_size=16)
    assert int(left) == 2


@pytest.mark.parametrize("shape,dtype", [((9, 16, 2, 64), torch.bfloat16), ((9, 3, 16, 65), torch.uint8),
                                         ((9, 2, 48, 72), torch.uint8), ((9, 3, 8, 128), torch.bfloat16),
                                         ((9, 4), torch.float32), ((9, 16, 64, 129), torch.uint8)])
def test_copy(ops, shape, dtype):
    g = torch.Generator().manual_seed(1)
    pools = [torch.randint(0, 256, (int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size(),), generator=g,
                           dtype=torch.uint8).view(dtype).view(shape).to(DEV) for _ in range(3)]
    before = [p.clone() for p in pools]
    err = i32([0])
    ops.copy_pages(pools, i32([0, -1, 4, 3, 7]), i32([8, 2, 1, -1, 7]), device_error=err)
    for p, b in zip(pools, before):
        want = b.view(torch.uint8).clone()
        want[8], want[1] = want[0].clone(), want[4].clone()
        assert torch.equal(p.view(torch.uint8), want)
    assert int(err) == 0


def test_copy_bad_ids_and_counts(ops):
    pool = torch.arange(6 * 16, dtype=torch.int32, device=DEV).view(6, 16)
    b, err = pool.clone(), i32([0])
    ops.copy_pages([pool], i32([0, 6, 1]), i32([3, 2, 1 << 30]), device_error=err)
    assert int(err) == 1 and torch.equal(pool[3], b[0]) and torch.equal(pool[2], b[2])
    for count, k in ((0, 0), (1, 1), (2, 2), (9, 2), (-1, 0)):
        q = b.clone()
        ops.copy_pages([q], i32([0, 1]), i32([4, 5]), count=i32([count]))
        want = b.clone()
        want[4:4 + k] = b[:k]
        assert torch.equal(q, want), count
    from paged_attention_relative_attn_gb300 import InklingError
    with pytest.raises(InklingError):
        ops.copy_pages([torch.zeros((4, 6), dtype=torch.int32, device=DEV)], i32([0]), i32([1]))  # 24 bytes a page


def test_copy_many_pools_and_offsets_past_32_bits(ops):
    """More pools than one launch takes; pools of more than 2^32 bytes."""
    pools = list(torch.arange(300 * 4 * 8, dtype=torch.int32, device=DEV).view(300, 4, 8))
    before = torch.stack(pools).clone()
    ops.copy_pages(pools, i32([0, 2]), i32([3, 1]))
    after = torch.stack(pools)
    assert torch.equal(after[:, 3], before[:, 0]) and torch.equal(after[:, 1], before[:, 2])
    assert torch.equal(after[:, ::2], before[:, ::2])
    n = (1 << 32) // (1 << 17) + 5
    big = torch.zeros((n, 1 << 17), dtype=torch.uint8, device=DEV)
    big[n - 2] = torch.arange(1 << 17, device=DEV).to(torch.uint8)
    ops.copy_pages([big], i32([n - 2, 5]), i32([n - 1, 2]))
    assert torch.equal(big[n - 1], big[n - 2]) and not big[2].any() and not big[:n - 2].any()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", ["q8", "q4", "bf16"])
def test_samples_of_a_prompt(ops, kind):
    """A prompt is prefilled once and forked; the samples decode on from the shared pages, some end, the pool is
    compacted, the others go on: every step as for requests that never shared anything."""
    B, H_q, H_kv, D, P, stride, R = 4, 4, 2, 64, 16, 8, 32
    g = torch.Generator().manual_seed(3)
    n_pages = 40
    rows = {"q8": (H_kv, P, 65), "q4": (H_kv, P, 36), "bf16": (P, H_kv, D)}[kind]

    def cache():
        dtype = torch.bfloat16 if kind == "bf16" else torch.uint8
        return [torch.zeros((n_pages, *rows), dtype=dtype, device=DEV) for _ in range(2)]

    class Run:
        def __init__(self):
            self.k, self.v = cache()
            self.lens, self.table = i32([0] * B), i32(np.zeros((B, stride), dtype=int))
            self.refs, self.free = i32([0] * n_pages), i32(np.random.default_rng(1).permutation(n_pages))
            self.count, self.err = i32([n_pages]), i32([0])

        def step(self, new, k, v, q, rel):
            _, cu, slots, _ = ops.build_tables(self.lens, i32(new), self.table, self.free, self.count, page_size=P,
                                               max_tokens=64, kv_lens=self.lens, free_left=self.count,
                                               device_error=self.err)
            if kind == "bf16":
                T = sum(max(x, 0) for x in new)
                ops.kv_append(k[:T].contiguous(), v[:T].contiguous(), cu, self.lens, self.table, self.k, self.v, device_error=self.err)
                return ops.decode(q, self.k, self.v, self.table, self.lens, rel, window=0, scale=0.125,
                                  max_seq_len=stride * P, device_error=self.err)
            append, decode = (getattr(ops, f"{name}_{kind}") for name in ("kv_append", "decode"))
            append(k, v, slots, self.k, self.v, device_error=self.err)
            return decode(q, self.k, self.v, self.table, self.lens, rel, window=0, scale=0.125, device_error=self.err)

    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    shared, apart = Run(), Run()
    k, v, q, rel = bf(64, H_kv, D), bf(64, H_kv, D), bf(B, H_q, D), torch.randn((B, H_q, R), generator=g).to(DEV)
    # one prompt of 41 tokens, and another request; apart: the prompt four times over
    shared.step([41, 0, 0, 0], k, v, q, rel)
    for b in range(B):
        new = [0] * B
        new[b] = 41
        apart.step(new, k, v, q, rel)
    _, src, dst, _ = ops.fork_pages(i32([-1, 0, 0, 0]), shared.lens, shared.table, shared.refs, shared.free,
                                    shared.count, page_size=P, kv_lens=shared.lens, free_left=shared.count,
                                    device_error=shared.err)
    ops.copy_pages([shared.k, shared.v], src, dst, device_error=shared.err)
    assert shared.lens.tolist() == [41] * 4 and int(shared.count) == n_pages - 3 - 3
    for t in range(12):
        if t == 5:  # samples 0 and 2 end
            new = i32([-1, 1, -1, 1])
            for r in (shared, apart):
                ops.release_pages(r.lens, new, r.table, r.refs, r.free, r.count, page_size=P, kv_lens=r.lens,
                                  free_left=r.count, device_error=r.err)
            assert int(shared.refs.sum()) == 2 and shared.lens.tolist() == [0, 46, 0, 46]
        if t == 8:
            s, d, moves = ops.compact_pages(shared.lens, shared.table, shared.free, shared.count, page_size=P,
                                            page_refs=shared.refs, device_error=shared.err)
            ops.copy_pages([shared.k, shared.v], s, d, count=moves, device_error=shared.err)
            used = {int(shared.table[b, c]) for b in (1, 3) for c in range(4 if int(shared.lens[b]) > 48 else 3)}
            assert used == set(range(len(used)))
        new = [1] * B if t < 5 else [0, 1, 0, 1]
        k, v, q, rel = bf(64, H_kv, D), bf(64, H_kv, D), bf(B, H_q, D), torch.randn((B, H_q, R), generator=g).to(DEV)
        (a, la), (b, lb) = shared.step(new, k, v, q, rel), apart.step(new, k, v, q, rel)
        assert torch.equal(a, b) and torch.equal(la, lb), t
    assert int(shared.err) == 0 and int(apart.err) == 0


def test_captured_fork_and_release(ops):
    """One captured step -- fork, copy, release, compact, copy -- replayed over states written in place."""
    P, stride, B = 16, 6, 6
    d = State([0] * B, P, stride, 30, 1).dev()
    source, new = i32([-1] * B), i32([1] * B)
    n = d["free"].numel()
    pool = torch.zeros((n, 64), dtype=torch.int32, device=DEV)
    bufs = [i32([0] * B) for _ in range(2)] + [i32([0] * n) for _ in range(2)] + [i32([0])]

    def step():
        ops.fork_pages(source, d["lens"], d["table"], d["refs"], d["free"], d["count"], page_size=P, kv_lens=d["lens"],
                       copy_src=bufs[0], copy_dst=bufs[1], free_left=d["count"])
        ops.copy_pages([pool], bufs[0], bufs[1])
        ops.release_pages(d["lens"], new, d["table"], d["refs"], d["free"], d["count"], page_size=P, kv_lens=d["lens"],
                          free_left=d["count"])
        ops.compact_pages(d["lens"], d["table"], d["free"], d["count"], page_size=P, page_refs=d["refs"],
                          move_src=bufs[2], move_dst=bufs[3], moves=bufs[4])
        ops.copy_pages([pool], bufs[2], bufs[3], count=bufs[4])

    step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for seed in range(5):
        rng = np.random.default_rng(seed)
        lens = list(rng.integers(1, 90, 3)) + [0, 0, 0]
        used = sum(pages_for(x, P) for x in lens)
        s = State(lens, P, stride, 30 - used, seed + 5)
        assert s.n_pages == n
        src = [-1, -1, -1] + [int(x) for x in rng.integers(-1, 3, 3)]
        nw = [int(x) for x in rng.choice([-1, 1], B)]
        for name, t in s.dev().items():
            d[name].copy_(t)
        source.copy_(i32(src))
        new.copy_(i32(nw))
        pool.copy_(torch.arange(n * 64, dtype=torch.int32, device=DEV).view(n, 64) + seed)
        data = pool.cpu().numpy().copy()
        gr.replay()
        f = ref_fork(src, s.lens, s.table, s.refs, s.free, s.count, P)
        for a, z in zip(f["src"], f["dst"]):
            if a >= 0:
                data[z] = data[a]
        r = ref_release(f["kv_lens"], nw, f["table"], f["refs"], s.free, f["left"], P)
        c = ref_compact(r["kv_lens"], f["table"], r["refs"], r["free"], r["left"], P)
        data[c["dst"][:c["moves"]]] = data[c["src"][:c["moves"]]]
        assert np.array_equal(d["table"].cpu().numpy(), c["table"]) and np.array_equal(d["free"].cpu().numpy(), c["free"])
        assert np.array_equal(d["refs"].cpu().numpy(), c["refs"]) and int(d["count"]) == r["left"]
        assert np.array_equal(pool.cpu().numpy(), data)


def test_on_another_stream_and_of_another_device(ops):
    from types import SimpleNamespace
    s = State([40, 0], 16, 4, 5, 3)
    d = s.dev()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pool = torch.arange(s.n_pages * 8, dtype=torch.int32, device=DEV).view(s.n_pages, 8)
    want = ref_fork([-1, 0], s.lens, s.table, s.refs, s.free, s.count, 16)
    kv, src, dst, left = ops.fork_pages(i32([-1, 0]), d["lens"], d["table"], d["refs"], d["free"], d["count"],
                                        page_size=16, stream=st)
    ops.copy_pages([pool], src, dst, stream=st)
    torch.cuda.synchronize()
    assert np.array_equal(kv.cpu().numpy(), want["kv_lens"]) and torch.equal(pool[int(dst[1])], pool[int(src[1])])
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0, device_index=1, stream_id=0, device_type=1)
    before = {k: v.clone() for k, v in d.items()}
    for call in (lambda: ops.fork_pages(i32([-1, 0]), d["lens"], d["table"], d["refs"], d["free"], d["count"], page_size=16, stream=other),
                 lambda: ops.release_pages(d["lens"], i32([-1, -1]), d["table"], d["refs"], d["free"], d["count"], page_size=16, stream=other),
                 lambda: ops.compact_pages(d["lens"], d["table"], d["free"], d["count"], page_size=16, stream=other),
                 lambda: ops.copy_pages([pool], src, dst, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(before[k], d[k]) for k in d)
