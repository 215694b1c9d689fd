"""The oracle's append writes the rows of its slots and no other byte of the pool."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.q4 as q4


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_other_places_keep_their_bytes(D, is_v):
    rng = np.random.default_rng(3)
    n, H, P = 3, 2, 32
    pool = rng.integers(0, 256, (n, H, P, 9 * D // 16), dtype=np.uint8)
    rows = torch.from_numpy(rng.standard_normal((6, H, D))).to(torch.bfloat16).double().numpy()
    slots = [0, 17, 31, 64, -1, n * P]
    out = q4.ref_append_q4(pool, rows, slots, is_v)
    # a place's bytes, by the definition: 16-place blocks of nibble rows, then scale rows
    mine = np.zeros((n, H, P // 16, 9 * D), dtype=bool)
    for slot in slots[:4]:
        page, place = divmod(slot, P)
        blk, r = divmod(place, 16)
        mine[page, :, blk, r * (D // 2):(r + 1) * (D // 2)] = True
        mine[page, :, blk, 8 * D + r * (D // 16):8 * D + (r + 1) * (D // 16)] = True
    mine = mine.reshape(pool.shape)
    assert mine.sum() == 4 * H * 9 * D // 16
    assert np.array_equal(out[~mine], pool[~mine]) and not np.array_equal(out[mine], pool[mine])
    # the rows written do not depend on what was there
    again = q4.ref_append_q4(255 - pool, rows, slots, is_v)
    assert np.array_equal(out[mine], again[mine])
