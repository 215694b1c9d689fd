"""Sizes at which the 8-bit rows' kernels take another form: windows of 1, 4 and 8 tokens, two heads per thread of a
read; and calls that the documentation allows between them."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.q8_cases import random_pool
from tests.test_q8_gpu import BF16, DEV, check_append, ops, runs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,starts,H,D,P", [
    ([70, 1, 1, 200, 33], [3, 15, 16, 30, 0], 16, 64, 32),    # 4880 rows: windows of 4
    ([1] * 300, [7 * i % 48 for i in range(300)], 15, 64, 48),
    ([1023, 1, 17], [5, 1, 14], 16, 64, 16),                  # 16656: windows of 8
    ([511, 1], [15, 0], 8, 128, 64),                          # 4096, the border
    ([2047, 1], [0, 9], 8, 64, 16),                           # 16384, the border
])
def test_append_windows(ops, counts, starts, H, D, P):  # noqa: F811
    g = torch.Generator().manual_seed(len(counts))
    slots, n = runs(counts, starts, P, g)
    T = slots.numel()
    pools = [random_pool(n, H, P, D, 5 + i, "cpu") for i in range(2)]
    k, v = (torch.randn((T, H, D), generator=g) * torch.exp(torch.randn((T, 1, 1), generator=g)) for _ in range(2))
    check_append(ops, k.to(BF16), v.to(BF16), slots, pools[0].to(DEV), pools[1].to(DEV), pools[0].numpy(),
                 pools[1].numpy())


def test_append_tokens_of_a_block_in_any_order_between_others(ops):  # noqa: F811
    """A block's tokens anywhere among 16 of the call: in reverse, and between tokens of other blocks and skipped
    ones."""
    H, D, P = 3, 128, 32
    g = torch.Generator().manual_seed(9)
    a, b, c = torch.arange(16) + 64, torch.arange(16) + 160, torch.arange(8) + 8
    slots = torch.cat([a.flip(0), torch.stack([b[:8], torch.full((8,), -1)], 1).flatten(), b[8:],
                       torch.stack([c, torch.arange(8) * 16 + 193], 1).flatten()])
    T = slots.numel()
    pools = [random_pool(12, H, P, D, 5 + i, "cpu") for i in range(2)]
    k, v = (torch.randn((T, H, D), generator=g).to(BF16) for _ in range(2))
    # (b's tokens lie within 24 of the call: as two calls)
    for i in (slice(0, 16), slice(16, 32), slice(32, 40), slice(40, 56)):
        got = [x.to(DEV) for x in pools]
        want = check_append(ops, k[i], v[i], slots[i], *got, pools[0].numpy(), pools[1].numpy())
        pools = [torch.from_numpy(x) for x in want]


@pytest.mark.parametrize("T,H,D", [(7000, 5, 128), (6600, 11, 64), (2049, 17, 128)])
def test_large_reads(ops, T, H, D):  # noqa: F811
    """Rows of a large read, heads odd, against those of small ones; slots repeat, some are negative."""
    P = 48
    g = torch.Generator().manual_seed(T)
    n = 60
    k, v = (random_pool(n, H, P, D, 3 + i, DEV) for i in range(2))
    slots = torch.randint(0, n * P, (T,), generator=g)
    slots[::97] = -1
    slots = slots.to(DEV)
    kr, vr = ops.kv_read_q8(slots, k, v)
    parts = [ops.kv_read_q8(s, k, v) for s in slots.split(500)]
    for got, i in ((kr, 0), (vr, 1)):
        want = torch.cat([x[i] for x in parts])
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert not kr[::97].any() and not vr[::97].any()


def test_decode_of_large_batches_reads_every_length(ops):  # noqa: F811
    """Batches around the 128 sequences whose lengths are looked at together."""
    from tests.q8_cases import check, make
    from tests.test_q8_gpu import run_decode
    for B in (127, 128, 129, 257):
        lens = [int(x) for x in np.random.default_rng(B).integers(0, 150, B)]
        inp = make([1] * B, lens, 4, 2, 64, 16, 60, 32, seed=B)
        check(inp, *run_decode(ops, inp, 1), what=str(B))
