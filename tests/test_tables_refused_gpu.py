"""A refused request's rows stay out of what the rest of a step does: every call that places or reads tokens by
length skips it when it is given ``step_lens``, and the request can ask again."""

from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
P, H, D, STRIDE, PAGES = 16, 2, 64, 3, 8


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def rows(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).to(DEV)


class Step:
    """Three requests of 16, 16 and 5 tokens ask for ``new`` more; the stack has one page, 7, so request 1 gets none."""

    def __init__(self, ops, new=(1, 1, 1), max_tokens=None, row=STRIDE):
        self.ops, self.new = ops, list(new)
        self.lens, self.pt = i32([16, 16, 5]), i32([[0, -1, -1], [1, -1, -1], [2, -1, -1]])[:, :row].contiguous()
        self.free, self.count = i32([7, 0, 0, 0, 0, 0, 0, 0]), i32([1])
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.step = torch.full((3,), -7, dtype=torch.int32, device=DEV)
        self.T = sum(new)
        self.kv, self.cu, self.slots, _ = ops.build_tables(
            self.lens, i32(new), self.pt, self.free, self.count, page_size=P, max_tokens=max_tokens or self.T,
            kv_lens=self.lens, free_left=self.count, step_lens=self.step, device_error=self.err)
        self.k, self.v = rows(self.T, H, D, seed=1), rows(self.T, H, D, seed=2)


def test_step_lens(ops):
    s = Step(ops)
    assert s.kv.tolist() == [17, 16, 6] and s.step.tolist() == [17, 0, 6] and int(s.err) == 32
    # all refusals, an ended request, one that asks for nothing
    step = torch.empty(5, dtype=torch.int32, device=DEV)
    kv, *_ = ops.build_tables(i32([30, 10, -4, 20, 7]), i32([3, 7, 1, -1, 0]), i32([[0, 1], [2, 3], [4, 5], [6, 0], [5, 0]]),
                              i32([7] + [0] * 9), i32([0]), page_size=16, max_tokens=20, step_lens=step)
    assert kv.tolist() == [30, 17, -4, 0, 7] and step.tolist() == [0, 17, 0, 0, 7]
    # the other outputs are what they are without it
    a = Step(ops)
    kv, cu, slots, left = ops.build_tables(i32([16, 16, 5]), i32([1, 1, 1]), i32([[0, -1, -1], [1, -1, -1], [2, -1, -1]]),
                                           i32([7] + [0] * 7), i32([1]), page_size=P, max_tokens=3)
    assert torch.equal(kv, a.kv) and torch.equal(cu, a.cu) and torch.equal(slots, a.slots) and torch.equal(left, a.count)


@pytest.mark.parametrize("new", [(1, 1, 1), (3, 14, 2)])
def test_kv_append_skips_it(ops, new):
    s = Step(ops, new)
    kc, vc = rows(PAGES, P, H, D, seed=3), rows(PAGES, P, H, D, seed=4)
    wk, wv = kc.clone(), vc.clone()
    ops.kv_append(s.k, s.v, s.cu, s.step, s.pt, kc, vc, device_error=s.err)
    for t, slot in enumerate(s.slots.tolist()):  # -1: the refused request's
        if slot >= 0:
            wk[slot // P, slot % P], wv[slot // P, slot % P] = s.k[t], s.v[t]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)  # request 1's last tokens among the untouched ones
    assert s.slots.tolist().count(-1) == new[1] and int(s.err) == 32 | 8


def test_kv_append_q4_skips_it(ops):
    s = Step(ops, (3, 14, 2))
    pool = torch.randint(0, 256, (PAGES, H, P, 9 * D // 16), dtype=torch.uint8, device=DEV)
    kc, vc = pool.clone(), pool.clone()
    ops.kv_append_q4(s.k, s.v, s.slots, kc, vc, device_error=s.err)
    assert torch.equal(kc[1], pool[1]) and torch.equal(vc[1], pool[1]) and int(s.err) == 32


@pytest.mark.parametrize("new", [(1, 1, 1), (3, 14, 2)])
def test_kv_conv_append_skips_it_and_its_state(ops, new):
    s = Step(ops, new)
    width = 4
    w = torch.randn((H, D, width), generator=torch.Generator().manual_seed(5)).to(DEV)
    st = [rows(3, width - 1, H, D, seed=6 + i) for i in range(2)]
    pools = [rows(PAGES, P, H, D, seed=8 + i) for i in range(2)]
    st0, pools0 = [x.clone() for x in st], [x.clone() for x in pools]
    which = i32([2, 0, 1])
    ops.kv_conv_append(s.k, s.v, s.cu, s.step, s.pt, pools[0], pools[1], w, w, st[0], st[1], which, max_q_len=max(new),
                       device_error=s.err)
    # the same without request 1
    keep = torch.tensor([t for t in range(s.T) if not new[0] <= t < new[0] + new[1]], device=DEV)
    ops.kv_conv_append(s.k[keep], s.v[keep], i32([0, new[0], new[0] + new[2]]), s.step[[0, 2]].contiguous(),
                       s.pt[[0, 2]].contiguous(), pools0[0], pools0[1], w, w, st0[0], st0[1], i32([2, 1]),
                       max_q_len=max(new))
    for got, want in zip(st + pools, st0 + pools0):
        assert torch.equal(got, want)
    assert int(s.err) == 32 | 8


def test_attention_skips_it(ops):
    s = Step(ops)
    q = rows(3, 4, D, seed=10)
    rel = torch.randn((3, 4, 8), generator=torch.Generator().manual_seed(11)).to(DEV)
    kc, vc = rows(PAGES, P, H, D, seed=12), rows(PAGES, P, H, D, seed=13)
    k4 = torch.zeros((PAGES, H, P, 9 * D // 16), dtype=torch.uint8, device=DEV)
    v4 = k4.clone()
    ops.kv_append_q4(kc.view(-1, H, D), vc.view(-1, H, D), torch.arange(PAGES * P, device=DEV), k4, v4)
    kw = dict(window=0, scale=0.1)
    for dec in (lambda lens: ops.decode(q, kc, vc, s.pt, lens, rel, max_seq_len=48, **kw),
                lambda lens: ops.decode_q4(q, k4, v4, s.pt, lens, rel, **kw)):
        out, lse = dec(s.step)
        want, wl = dec(s.kv)
        assert torch.equal(out[[0, 2]], want[[0, 2]]) and torch.equal(lse[[0, 2]], wl[[0, 2]])
        assert not out[1].any() and bool((lse[1] == -float("inf")).all())
    for pre in (lambda lens, out: ops.prefill(q, s.cu, kc, vc, s.pt, lens, rel, max_seq_len=48, max_q_len=1, out=out, **kw),
                lambda lens, out: ops.prefill_q4(q, s.cu, k4, v4, s.pt, lens, rel, max_seq_len=48, max_q_len=1, out=out, **kw)):
        out, _ = pre(s.step, torch.full_like(q, 7.0))
        want, _ = pre(s.kv, torch.full_like(q, 7.0))
        assert torch.equal(out[[0, 2]], want[[0, 2]]) and bool((out[1] == 7.0).all())


def test_it_asks_again(ops):
    """Refused, then served once a request has ended: its row ends up as if it had never been refused."""
    s = Step(ops)
    kc, vc = rows(PAGES, P, H, D, seed=3), rows(PAGES, P, H, D, seed=4)
    held = kc[1].clone()
    ops.kv_append(s.k, s.v, s.cu, s.step, s.pt, kc, vc)
    k2, v2 = rows(1, H, D, seed=20), rows(1, H, D, seed=21)
    new = i32([-1, 1, 0])
    _, cu, slots, left = ops.build_tables(s.lens, new, s.pt, s.free, s.count, page_size=P, max_tokens=1, kv_lens=s.lens,
                                          free_left=s.count, step_lens=s.step, device_error=s.err)
    assert s.lens.tolist() == [0, 17, 6] and s.step.tolist() == [0, 17, 6] and s.pt[1].tolist() == [1, 7, -1]
    ops.kv_append(k2, v2, cu, s.step, s.pt, kc, vc)
    assert torch.equal(kc[1], held) and torch.equal(kc[7, 0], k2[0]) and slots.tolist() == [7 * P]


def test_captured(ops):
    """In a captured step the refusal is decided on the device, replay by replay."""
    lens, pt, free, count = i32([15, 15]), i32([[0, -1], [1, -1]]), i32([3, 0, 0, 0]), i32([1])
    step, new = torch.empty(2, dtype=torch.int32, device=DEV), i32([1, 1])
    cu, slots = torch.empty(3, dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int64, device=DEV)
    kc, vc = torch.zeros((4, P, H, D), dtype=BF16, device=DEV), torch.zeros((4, P, H, D), dtype=BF16, device=DEV)
    k = torch.ones((2, H, D), dtype=BF16, device=DEV)
    start = [x.clone() for x in (lens, pt, free, count)]

    def go():
        ops.build_tables(lens, new, pt, free, count, page_size=P, kv_lens=lens, cu_seqlens_q=cu, slot_map=slots,
                         free_left=count, step_lens=step)
        ops.kv_append(k, k, cu, step, pt, kc, vc)

    go()
    for x, y in zip((lens, pt, free, count), start):
        x.copy_(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for i, want in enumerate(([16, 16], [17, 0], [18, 0])):
        k.fill_(float(i + 2))
        g.replay()
        assert step.tolist() == want, i
    assert lens.tolist() == [18, 16]
    assert bool((kc[1, 15] == 2.0).all()) and bool((kc[3, 1] == 4.0).all())


def test_too_few_slots_and_rows(ops):
    """Refused for slots: the caller's rows end before the packing does, and the appends leave its cache alone."""
    s = Step(ops, (3, 4, 2), max_tokens=5)  # rows 0..4: request 1's last two rows and request 2's are not there
    assert s.kv.tolist() == [19, 16, 5] and s.step.tolist() == [19, 0, 0] and int(s.err) == 8
    kc, vc = rows(PAGES, P, H, D, seed=3), rows(PAGES, P, H, D, seed=4)
    wk, wv = kc.clone(), vc.clone()
    k, v = s.k[:5].contiguous(), s.v[:5].contiguous()
    ops.kv_append(k, v, s.cu, s.step, s.pt, kc, vc)
    for t, slot in enumerate(s.slots.tolist()):
        if slot >= 0:
            wk[slot // P, slot % P], wv[slot // P, slot % P] = k[t], v[t]
    assert torch.equal(kc, wk) and torch.equal(vc, wv) and s.slots.tolist().count(-1) == 2
    width = 3
    w = torch.randn((H, D, width), generator=torch.Generator().manual_seed(5)).to(DEV)
    st = [rows(3, width - 1, H, D, seed=6 + i) for i in range(2)]
    before = [x.clone() for x in st]
    pools = [rows(PAGES, P, H, D, seed=8 + i) for i in range(2)]
    old = [x.clone() for x in pools]
    ops.kv_conv_append(k, v, s.cu, s.step, s.pt, pools[0], pools[1], w, w, st[0], st[1], i32([0, 1, 2]), max_q_len=4)
    for x, y in zip(st, before):
        assert torch.equal(x[1:], y[1:]) and not torch.equal(x[0], y[0])
    for x, y in zip(pools, old):
        assert torch.equal(x[[1, 2]], y[[1, 2]]) and not torch.equal(x[7], y[7])


def test_convolved_rows_for_the_4_bit_cache(ops):
    """The convolution into a staging pool, whose lengths are the step's new tokens and 0 for a refused request, then the
    4-bit append by slot: the refused request keeps its state and its rows."""
    new = (1, 14, 2)
    s = Step(ops, new)
    width = 4
    w = torch.randn((H, D, width), generator=torch.Generator().manual_seed(5)).to(DEV)
    st = [rows(3, width - 1, H, D, seed=6 + i) for i in range(2)]
    before = [x.clone() for x in st]
    stage = [torch.zeros((3, P, H, D), dtype=BF16, device=DEV) for _ in range(2)]
    mine = torch.where(s.step > 0, i32(new), 0).to(torch.int32)
    ops.kv_conv_append(s.k, s.v, s.cu, mine, i32([[0], [1], [2]]), stage[0], stage[1], w, w, st[0], st[1], i32([0, 1, 2]),
                       max_q_len=14)
    pool = torch.randint(0, 256, (PAGES, H, P, 9 * D // 16), dtype=torch.uint8, device=DEV)
    kc, vc = pool.clone(), pool.clone()
    at = torch.cat([torch.arange(n, device=DEV) + b * P for b, n in enumerate(new)])  # the rows' places in the staging pool
    ops.kv_append_q4(stage[0].view(-1, H, D)[at], stage[1].view(-1, H, D)[at], s.slots, kc, vc)
    for x, y in zip(st, before):
        assert torch.equal(x[1], y[1]) and not torch.equal(x[0], y[0]) and not torch.equal(x[2], y[2])
    assert torch.equal(kc[1], pool[1]) and torch.equal(vc[1], pool[1]) and not torch.equal(kc[7], pool[7])
