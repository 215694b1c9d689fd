"""Guard regions around everything that the calls on the 8-bit cache and on shared pages write: a byte before or behind
a buffer that changes is found, and so is an element that a call leaves out."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.q8 as q8
from oracle.pages import ref_compact, ref_fork, ref_release
from tests.helpers import f64
from tests.q8_cases import BF16 as P_BF16
from tests.q8_cases import check, make, random_pool, reference
from tests.test_guards_gpu import Guarded, ops  # noqa: F401 (ops: a fixture)
from tests.test_pages_gpu import State

pytestmark = pytest.mark.gpu
DEV = "cuda"


def guarded(t):
    """A copy of a tensor within guards."""
    g = Guarded(tuple(t.shape), t.dtype, fill=None)
    g.t.copy_(t)
    return g


def ints(a):
    return guarded(torch.tensor(np.asarray(a), dtype=torch.int32))


def unset(*shape):
    return Guarded(shape, torch.int32, fill=-77)


@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (37, 3, 128, 48), (700, 7, 64, 32), (1030, 16, 128, 16)])
def test_append_and_read(ops, T, H, D, P):  # noqa: F811
    """The first and the last block of the pools are among those written."""
    g = torch.Generator().manual_seed(T)
    n = (T + P - 1) // P + 1
    pools = [random_pool(n, H, P, D, 3 + i, "cpu") for i in range(2)]
    slots = torch.cat([torch.arange(T // 2), n * P - (T - T // 2) + torch.arange(T - T // 2)])
    k, v = (torch.randn((T, H, D), generator=g).to(torch.bfloat16) for _ in range(2))
    kc, vc = (guarded(x) for x in pools)
    rows = [Guarded((T, H, D), torch.bfloat16) for _ in range(2)]
    ops.kv_append_q8(k.to(DEV), v.to(DEV), slots.to(DEV), kc.t, vc.t)
    ops.kv_read_q8(slots.to(DEV), kc.t, vc.t, k_rows=rows[0].t, v_rows=rows[1].t)
    torch.cuda.synchronize()
    assert all(x.intact() for x in (kc, vc, *rows))
    for got, pool, x, is_v in ((kc, pools[0], k, False), (vc, pools[1], v, True)):
        want = q8.ref_append_q8(pool.numpy(), f64(x), slots.numpy(), is_v)
        assert np.array_equal(got.t.cpu().numpy(), want)
        read = q8.read_pool(want, is_v)[slots.numpy() // P, slots.numpy() % P]
        assert np.array_equal(f64(rows[is_v].t), read)


@pytest.mark.parametrize("q_len,lens,H_q,H_kv,D,P,window,R", [
    (1, [37, 100], 4, 2, 64, 16, 32, 32),
    (1, [5000, 20, 0, 1300], 12, 2, 128, 64, 0, 64),
    (4, [600, 64, 515, 4, 3], 6, 2, 128, 64, 512, 512),
    (7, [900, 133], 16, 1, 128, 64, 0, 33),
    (64, [64, 700], 4, 4, 64, 32, 100, 128),
])
def test_decode(ops, q_len, lens, H_q, H_kv, D, P, window, R):  # noqa: F811
    inp = make([q_len] * len(lens), lens, H_q, H_kv, D, P, window, R, seed=400 + q_len)
    out, lse = Guarded(tuple(inp.q.shape), torch.bfloat16), Guarded(tuple(inp.q.shape[:2]), torch.float32)
    need = ops.decode_q8_workspace_bytes(len(lens), q_len, H_q, H_kv, D)
    ws = Guarded((max(need, 16),), torch.uint8, fill=255)
    ops.decode_q8(inp.q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens, inp.rel_logits, q_len=q_len,
                  window=window, scale=inp.scale, out=out.t, lse=lse.t, workspace=ws.t)
    torch.cuda.synchronize()
    assert out.intact() and lse.intact() and ws.intact()
    check(inp, out.t, lse.t)


@pytest.mark.parametrize("q_lens,lens,H_q,H_kv,D,P,window,R", [
    ([130, 1, 255], [130, 70, 1000], 6, 2, 128, 64, 64, 64),
    ([77, 300], [1000, 300], 4, 1, 64, 16, 0, 32),
    ([128, 256], [128, 900], 6, 2, 128, 48, 512, 256),
])
def test_prefill(ops, q_lens, lens, H_q, H_kv, D, P, window, R):  # noqa: F811
    inp = make(q_lens, lens, H_q, H_kv, D, P, window, R, seed=420)
    spare = 9  # rows of no sequence
    q, rel = (torch.cat([x, x[:spare]]) for x in (inp.q, inp.rel_logits))
    T = inp.q.shape[0]
    out, lse = Guarded(tuple(q.shape), torch.bfloat16, fill=7.0), Guarded(tuple(q.shape[:2]), torch.float32, fill=7.0)
    need = ops.prefill_q8_workspace_bytes(len(lens), max(q_lens), H_kv, D, window, max(lens))
    ws = Guarded((need,), torch.uint8, fill=255)
    ops.prefill_q8(q, inp.cu_seqlens_q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens, rel, window=window,
                   scale=inp.scale, max_seq_len=max(lens), max_q_len=max(q_lens), out=out.t, lse=lse.t, workspace=ws.t)
    torch.cuda.synchronize()
    assert out.intact() and lse.intact() and ws.intact()
    assert bool((out.t[T:] == 7.0).all()) and bool((lse.t[T:] == 7.0).all())
    check(inp, out.t[:T], lse.t[:T], ref=reference(inp), p_step=P_BF16)


@pytest.mark.parametrize("B,P", [(3, 16), (33, 48), (300, 16)])
def test_pages(ops, B, P):  # noqa: F811
    """Fork, release and compaction in turn; pools just large enough, tables without a spare row or column."""
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 12 * P, B)
    lens[B // 2:] = 0
    kids = B - B // 2
    s = State(list(lens), P, 12, kids, B, nobody=0)
    source = np.full(B, -1)
    source[B // 2:] = rng.integers(0, B // 2, kids)
    table, refs, free, count, held = ints(s.table), ints(s.refs), ints(s.free), ints([s.count]), ints(s.lens)
    kv, src, dst, left = unset(B), unset(B), unset(B), unset(1)
    ops.fork_pages(ints(source).t, held.t, table.t, refs.t, free.t, count.t, page_size=P, kv_lens=kv.t, copy_src=src.t,
                   copy_dst=dst.t, free_left=left.t)
    f = ref_fork(source, s.lens, s.table, s.refs, s.free, s.count, P)
    every = [table, refs, free, count, held, kv, src, dst, left]
    same = lambda g, want: np.array_equal(g.t.cpu().numpy(), want)  # noqa: E731
    torch.cuda.synchronize()
    assert all(x.intact() for x in every)
    assert same(kv, f["kv_lens"]) and same(src, f["src"]) and same(dst, f["dst"]) and same(left, [f["left"]])
    assert same(table, f["table"]) and same(refs, f["refs"]) and same(free, s.free) and same(held, s.lens)
    new = np.where(rng.random(B) < 0.5, -1, 1)
    kv2, left2 = unset(B), unset(1)
    ops.release_pages(kv.t, ints(new).t, table.t, refs.t, free.t, left.t, page_size=P, kv_lens=kv2.t, free_left=left2.t)
    r = ref_release(f["kv_lens"], new, f["table"], f["refs"], s.free, f["left"], P)
    torch.cuda.synchronize()
    assert all(x.intact() for x in (*every, kv2, left2))
    assert same(kv2, r["kv_lens"]) and same(refs, r["refs"]) and same(free, r["free"]) and same(left2, [r["left"]])
    a, z, moves = unset(s.n_pages), unset(s.n_pages), unset(1)
    ops.compact_pages(kv2.t, table.t, free.t, left2.t, page_size=P, page_refs=refs.t, move_src=a.t, move_dst=z.t,
                      moves=moves.t)
    c = ref_compact(r["kv_lens"], f["table"], r["refs"], r["free"], r["left"], P)
    torch.cuda.synchronize()
    assert all(x.intact() for x in (*every, kv2, left2, a, z, moves))
    assert same(table, c["table"]) and same(refs, c["refs"]) and same(free, c["free"])
    assert same(a, c["src"]) and same(z, c["dst"]) and same(moves, [c["moves"]])


@pytest.mark.parametrize("page_bytes", [16, 4096 + 16, 32768, 32768 + 16, 100000 // 16 * 16, 131072])
def test_copy(ops, page_bytes):  # noqa: F811
    """The first and the last page of the pools, whole and in parts of odd sizes."""
    g = torch.Generator().manual_seed(page_bytes)
    data = [torch.randint(0, 256, (5, page_bytes), generator=g, dtype=torch.uint8) for _ in range(3)]
    pools = [guarded(x) for x in data]
    ops.copy_pages([p.t for p in pools], ints([0, 3]).t, ints([4, 1]).t)
    torch.cuda.synchronize()
    for p, x in zip(pools, data):
        want = x.clone()
        want[4], want[1] = x[0], x[3]
        assert p.intact() and torch.equal(p.t.cpu(), want)
