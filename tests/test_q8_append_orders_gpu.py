"""8-bit appends whose blocks' tokens lie in any order among 16 of the call, between tokens of other blocks and skipped
ones, at the sizes of each window (1, 4 and 8 tokens): byte for byte against the oracle."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.q8_cases import random_pool
from tests.test_q8_gpu import check_append, ops, special_rows  # noqa: F401 (ops: a fixture)

pytestmark = pytest.mark.gpu


def mixed_slots(T, blocks, seed):
    """Slots of T tokens: 16 tokens at a time, with gaps between, belong to up to four blocks that no other tokens have."""
    rng = np.random.default_rng(seed)
    ids = list(rng.permutation(blocks))
    out = []
    while len(out) < T:
        out += [-1] * int(rng.integers(0, 4))
        of = [ids.pop() for _ in range(int(rng.integers(1, 5)))]
        places = {b: list(rng.permutation(16)) for b in of}
        if rng.random() < 0.3:
            places[of[0]] = list(range(15, -1, -1))  # in order
        elif rng.random() < 0.3:
            places[of[0]] = list(range(16))          # in reverse
        for _ in range(16):
            b = of[int(rng.integers(len(of)))]
            out.append(-1 if rng.random() < 0.15 else int(b) * 16 + int(places[b].pop()))
    return np.array(out[:T])


@pytest.mark.parametrize("T,H,D,P", [(300, 2, 64, 32), (300, 3, 128, 16), (700, 7, 64, 48), (800, 6, 128, 64),
                                     (1100, 16, 64, 16), (1033, 16, 128, 256)])
def test_any_order_between_others(ops, T, H, D, P):  # noqa: F811
    per = P // 16
    pages = (4 * T // 16 + 8 + per - 1) // per
    slots = mixed_slots(T, pages * per, T)
    leads = {int(np.flatnonzero(slots // 16 == b)[0]) % 8 for b in np.unique(slots[slots >= 0] // 16)}
    assert leads == set(range(8))  # a block's first token at every place of a window
    pools = [random_pool(pages, H, P, D, 5 + i, "cpu") for i in range(2)]
    got = [x.to("cuda") for x in pools]
    want = [x.numpy() for x in pools]
    slots = torch.from_numpy(slots)
    want = check_append(ops, special_rows(T, H, D, 1), special_rows(T, H, D, 2), slots, *got, *want)
    g = torch.Generator().manual_seed(T)
    k, v = ((torch.randn((T, H, D), generator=g) * 2.0 ** 9).to(torch.bfloat16) for _ in range(2))
    check_append(ops, k, v, slots, *got, *want)  # larger: what stays in a block is rounded again
