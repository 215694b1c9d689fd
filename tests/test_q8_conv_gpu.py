"""The short convolution on the way into the 8-bit cache, and its state of requests that are forked."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.q8 as q8
from tests.helpers import f64

pytestmark = pytest.mark.gpu
DEV, BF16 = "cuda", torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


class Cache:
    """Requests of up to B rows over an 8-bit cache, their K and V convolved first, in a staging pool of the step's rows."""
    H, D, P, width, stride, n = 2, 64, 16, 4, 5, 24

    def __init__(self, ops, B, w):
        self.ops, self.B, self.w = ops, B, w
        self.k = torch.zeros((self.n, self.H, self.P, self.D + 1), dtype=torch.uint8, device=DEV)
        self.v = torch.zeros_like(self.k)
        self.lens, self.count, self.err = i32(*[0] * B), i32(self.n), i32(0)
        self.table = torch.zeros((B, self.stride), dtype=torch.int32, device=DEV)
        self.refs, self.free = torch.zeros(self.n, dtype=torch.int32, device=DEV), torch.randperm(self.n).to(DEV, torch.int32)
        # a row for each request: what it holds of both states goes with its row's number
        self.state = [torch.zeros((B, self.width - 1, self.H, self.D), dtype=BF16, device=DEV) for _ in range(2)]

    def step(self, new, k, v):
        """new[b] tokens of row b; returns the staged rows and the slots of the packed tokens."""
        new = i32(*new)
        _, cu, slots, _ = self.ops.build_tables(self.lens, new, self.table, self.free, self.count, page_size=self.P,
                                                max_tokens=k.shape[0], kv_lens=self.lens, free_left=self.count,
                                                device_error=self.err)
        per = 3  # pages of the staging pool for a request
        stage = [torch.zeros((self.B * per, self.P, self.H, self.D), dtype=BF16, device=DEV) for _ in range(2)]
        at = torch.arange(self.B * per, dtype=torch.int32, device=DEV).view(self.B, per)
        self.ops.kv_conv_append(k, v, cu, new, at, *stage, self.w, self.w, *self.state,
                                torch.arange(self.B, dtype=torch.int32, device=DEV), max_q_len=per * self.P,
                                device_error=self.err)
        # packed token i of request b is staged at place i of its pages
        first = cu[:-1].long().repeat_interleave(new.long())
        row = torch.arange(self.B, device=DEV).repeat_interleave(new.long())
        place = row * per * self.P + torch.arange(k.shape[0], device=DEV) - first
        rows = [s.view(-1, self.H, self.D)[place] for s in stage]
        self.ops.kv_append_q8(*rows, slots, self.k, self.v, device_error=self.err)
        return rows, slots


def rows_of(g, T):
    return [torch.randn((T, Cache.H, Cache.D), generator=g).to(BF16).to(DEV) for _ in range(2)]


def test_convolved_rows_through_a_staging_pool(ops):
    g = torch.Generator().manual_seed(7)
    c = Cache(ops, 3, torch.randn((Cache.H, Cache.D, Cache.width), generator=g).to(DEV))
    want = [np.zeros(tuple(c.k.shape), dtype=np.uint8) for _ in range(2)]
    for new in ([1, 20, 5], [1, 1, 1], [7, 1, 30], [1, 1, 1]):
        rows, slots = c.step(new, *rows_of(g, sum(new)))
        for i, (pool, is_v) in enumerate(((c.k, False), (c.v, True))):
            want[i] = q8.ref_append_q8(want[i], f64(rows[i]), slots.cpu().numpy(), is_v)
            assert np.array_equal(pool.cpu().numpy(), want[i])
    assert int(c.err) == 0


def test_state_of_forked_requests(ops):
    """Two samples go on from a prompt: the full pages shared, the last page and the state's rows copied.  Each then has
    in the cache what it has if its prompt was its own."""
    g = torch.Generator().manual_seed(8)
    w = torch.randn((Cache.H, Cache.D, Cache.width), generator=g).to(DEV)
    shared, apart = Cache(ops, 3, w), Cache(ops, 3, w)
    k, v = rows_of(g, 37)
    shared.step([37, 0, 0], k, v)
    for b in range(3):
        apart.step([37 if i == b else 0 for i in range(3)], k, v)
    s = shared
    _, src, dst, _ = ops.fork_pages(i32(-1, 0, 0), s.lens, s.table, s.refs, s.free, s.count, page_size=s.P,
                                    kv_lens=s.lens, free_left=s.count, device_error=s.err)
    ops.copy_pages([s.k, s.v], src, dst, device_error=s.err)
    ops.copy_pages(s.state, i32(0, 0), i32(1, 2), device_error=s.err)  # a state's row is a page of its pool
    assert s.lens.tolist() == [37] * 3 and s.refs.sum() == 4
    for new in ([1, 1, 1], [4, 1, 12], [1, 1, 1]):
        k, v = rows_of(g, sum(new))
        for c in (shared, apart):
            c.step(new, k, v)
    assert torch.equal(shared.lens, apart.lens) and int(shared.err) == int(apart.err) == 0
    for b in range(3):
        at = torch.arange(int(shared.lens[b]), device=DEV)
        read = [ops.kv_read_q8(c.table[b].long()[at // c.P] * c.P + at % c.P, c.k, c.v) for c in (shared, apart)]
        assert torch.equal(read[0][0], read[1][0]) and torch.equal(read[0][1], read[1][1])
    for a, z in zip(shared.state, apart.state):
        assert torch.equal(a, z)
